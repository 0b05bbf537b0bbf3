"""8-bit paged cache: one scale per (block, kv head) for K and for V.  Test infrastructure only.

The quantizer follows a stated float32 op sequence, so its codes are bit-exact by construction:
big = max |x| over the rows the block holds; scale = big * (1 / M) and inv = (1 / big) * M, each
operation in float32 (both 0 when big < 2^-110); code = x * inv in float32, rounded to the format (nearest even): e4m3 with
saturation (M = 448), or integers in [-127, 127] (M = 127).  The value held is code * scale.
"""
import numpy as np

MOST = {"e4m3": 448.0, "int8": 127.0}


def round_e4m3(y):
    """Nearest-even rounding of float values to e4m3 (4 exponent bits, bias 7, 3 mantissa bits, largest
    448, subnormal step 2^-9), saturating; NaN stays NaN."""
    y = np.asarray(y, dtype=np.float64)
    a = np.abs(y)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    r = np.minimum(np.round(a / step) * step, 448.0)
    return np.copysign(r, y)


def quantize_rows(x, fmt):
    """(codes as float64 values, scale as float32) of one group (any shape)."""
    x = np.asarray(x, dtype=np.float32)
    big = np.float32(np.abs(x).max()) if x.size else np.float32(0)
    if not big >= np.float32(2.0 ** -110):
        return np.zeros(x.shape), np.float32(0)
    m = np.float32(MOST[fmt])
    one = np.float32(1)
    scale, inv = np.float32(big * np.float32(one / m)), np.float32(np.float32(one / big) * m)
    y = (x * inv).astype(np.float32)
    if fmt == "e4m3":
        return round_e4m3(y), scale
    return np.clip(np.round(y.astype(np.float64)), -127, 127), scale


class Q8Cache:
    """The cache as a function of what was appended: per (block, kv head) the bf16 rows held, from
    which codes and scales follow."""

    def __init__(self, num_blocks, n_kv, block_size, head_dim, fmt):
        self.fmt, self.bs = fmt, block_size
        self.rows = np.zeros((2, num_blocks, n_kv, block_size, head_dim))
        self.codes = np.zeros_like(self.rows)
        self.scales = np.zeros((num_blocks, n_kv, 2), dtype=np.float32)

    def append(self, k, v, slots):
        touched = set()
        for i, slot in enumerate(np.asarray(slots).tolist()):
            if slot < 0:
                continue
            b, r = divmod(int(slot), self.bs)
            if r == 0:
                self.rows[:, b] = 0.0                          # a block taken anew
            self.rows[0, b, :, r], self.rows[1, b, :, r] = k[i], v[i]
            touched.add((b, r))
        last = {}
        for b, r in touched:
            last[b] = max(last.get(b, 0), r)
        for b, r in last.items():
            for g in range(self.rows.shape[2]):
                for i in range(2):
                    c, s = quantize_rows(self.rows[i, b, g, :r + 1], self.fmt)
                    self.codes[i, b, g] = 0.0
                    self.codes[i, b, g, :r + 1] = c
                    self.scales[b, g, i] = s

    def values(self):
        """K and V held, float64 [num_blocks][n_kv][bs][d]."""
        s = self.scales.astype(np.float64)
        return self.codes[0] * s[:, :, 0, None, None], self.codes[1] * s[:, :, 1, None, None]
