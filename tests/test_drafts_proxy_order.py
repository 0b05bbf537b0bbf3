"""Attention of drafted tokens, read from the source (no GPU): what the softmax warps write into shared memory that TMA loads
write next is fenced behind their last access, before the slot is given away."""
import re

from test_coherent_loads import kernels, source


def test_the_scratch_of_a_tile_is_fenced_before_its_slot_is_given_away():
    body = next(b for n, _, b in kernels(source("decode_rows.cu")) if n == "decode_rows_kernel")
    given = body.index("mbar_arrive(&sh.pfull[pb])")
    # accesses of the scratch behind P, from the last pass over the tile on
    used = [m.end() for m in re.finditer(r"scr\.(red|factor|win|seen)", body[:given])]
    assert used and not re.search(r"scr\.", body[given:])
    fences = [m.start() for m in re.finditer(r"fence_proxy_async_smem\(\);", body[:given])]
    assert fences[-1] > used[-1], "the sums of a segment's end are written behind the last fence"
    # by every thread: the fence stands in no branch of one thread or warp, and no barrier is missing ahead of it
    between = body[used[-1]:fences[-1]]
    assert between.count("{") == between.count("}") and "if (lane" not in between and "elected" not in between
    assert "sync(false)" in body[fences[-2]:used[-1]]
