"""Outputs and workspaces of the attention of drafted tokens that overlap what the call still reads are refused, before anything
is used (no GPU)."""
import ctypes

import pytest

from test_drafts_host import EINVAL, latent, tree

T, B, H, KV, D, BS, NB, MB, W = 6, 3, 8, 2, 128, 16, 9, 4, 2
MIB = 1 << 20
LAT, ROPE = 512, 64
# argument: (address, bytes), apart from one another
KEYS = dict(q=(MIB, T * H * D * 2), k=(2 * MIB, NB * KV * BS * D * 2), v=(3 * MIB, NB * KV * BS * D * 2), bt=(4 * MIB, B * MB * 4), ctx=(5 * MIB, B * 4),
            start=(6 * MIB, (B + 1) * 4), mask=(7 * MIB, T * W * 8), err=(8 * MIB, 4))
LATENT = dict(KEYS, q=(MIB, T * H * (LAT + ROPE) * 2), cache=(2 * MIB, NB * BS * (LAT + ROPE) * 2))
del LATENT["k"], LATENT["v"]
OUT, WS = 32 * MIB, 64 * MIB


def args(places, **k):
    return {n: ctypes.c_void_p(a) for n, (a, _) in places.items()} | dict(words=W, out=ctypes.c_void_p(OUT), ws=ctypes.c_void_p(WS)) | k


@pytest.mark.parametrize("call,places,v", [(tree, KEYS, D), (latent, LATENT, LAT)], ids=["tree", "latent"])
@pytest.mark.parametrize("kind", [0, 1])
def test_an_output_over_an_input(call, places, v, kind):
    size = T * H * v * (4 if kind else 2)
    for name, (at, n) in places.items():
        for out in (at, (at + n - 1) // 16 * 16, at + 16 - size):
            assert call(**args(places, kind=kind, out=ctypes.c_void_p(out))) == EINVAL, (name, out)
    assert call(**args(places, kind=kind, out=ctypes.c_void_p(WS))) == EINVAL


@pytest.mark.parametrize("call,places", [(tree, KEYS), (latent, LATENT)], ids=["tree", "latent"])
def test_a_workspace_over_an_input(call, places):
    for name, (at, n) in places.items():
        for ws in (at, (at + n - 1) // 256 * 256):
            assert call(**args(places, ws=ctypes.c_void_p(ws))) == EINVAL, name


@pytest.mark.parametrize("call,places", [(tree, KEYS), (latent, LATENT)], ids=["tree", "latent"])
def test_apart_from_one_another_they_are_taken(call, places):
    # as far as a machine without a GPU goes; where there is one, nothing is run on made-up addresses
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    assert call(**args(places)) not in (0, EINVAL)
