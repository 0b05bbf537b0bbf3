"""RoPE re-rotation of reused key chunks.  Test infrastructure only.

Source: "Research Paper Review : CACHE BLEND, Fast Large Language Model Serving
for RAG with Cached Knowledge Fusion", section "Background" (full KV reuse): a
chunk's K/V are precomputed as if the chunk started at position 0; because RoPE
only encodes relative position, the chunk's keys are brought to their real
place by one extra rotation by (real start - 0), applied to every key of the
chunk alike.

Readings (the page names RoPE but not its pairing, base or precision):
rotate pairs (j, j + d/2) for j < d/2 by the angle delta * base^(-2j/d),
base 10000 by default; the oracle works in float64 and rounds the stored key
to bf16 (nearest even) once at the end.
"""
import numpy as np

from .rounding import round_bf16


def rotate(x, delta, base=10000.0):
    """Rotate the last axis of x (float64, length d) by position delta; no rounding."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    half = d // 2
    theta = float(delta) * np.power(float(base), -2.0 * np.arange(half) / d)
    c, s = np.cos(theta), np.sin(theta)
    x1, x2 = x[..., :half], x[..., half:]
    return np.concatenate([x1 * c - x2 * s, x1 * s + x2 * c], axis=-1)


def rope_shift_k(k_pool, block_ids, deltas, base=10000.0):
    """Return a copy of k_pool [num_blocks][n_kv][bs][d] with the listed blocks re-rotated.

    Block block_ids[i] (every kv head, every row) is rotated by deltas[i]; ids are
    distinct.  The result is rounded to bf16 values (float64 array).
    """
    kp = np.array(k_pool, dtype=np.float64, copy=True)
    for b, dl in zip(np.asarray(block_ids).tolist(), np.asarray(deltas).tolist()):
        kp[int(b)] = round_bf16(rotate(kp[int(b)], dl, base))
    return kp


def rope_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """(angle per position of each channel pair, multiplier of cos and sin) after a scaling for
    contexts `factor` times the trained length, float64.

    none; linear: every angle divided by factor; ntk: base * factor^(r / (r - 2)); parts: pairs
    that make at least `high` turns over the trained length keep their angle, those with at most
    `low` turns are divided by factor, between them the share is linear in the turns; yarn: the
    share is linear in the pair's index, between the (rounded) indices whose turns are high and
    low, and cos and sin are multiplied by 0.1 ln(factor) + 1.
    """
    r = rotary_dim
    out, amp = [], 1.0
    b = base * factor ** (r / (r - 2.0)) if scaling == "ntk" else base
    if scaling == "yarn":
        index = [r * np.log(original_len / (2 * np.pi * t)) / (2 * np.log(b)) for t in (high, low)]
        i0, i1 = max(np.floor(index[0]), 0), min(np.ceil(index[1]), r - 1)
        amp = 0.1 * np.log(factor) + 1.0
    for j in range(r // 2):
        w = 1.0 / b ** (2.0 * j / r)
        keep = 1.0
        if scaling == "linear":
            keep = 0.0
        elif scaling == "parts":
            keep = (original_len * w / (2 * np.pi) - low) / (high - low)
        elif scaling == "yarn":
            keep = 1.0 - (j - i0) / max(i1 - i0, 0.001)
        keep = min(max(keep, 0.0), 1.0)
        out.append(keep * w + (1.0 - keep) * w / factor)
    return np.array(out), amp


def rope_tokens(x, positions, freqs, amp=1.0, interleaved=False):
    """Rotate the first 2 len(freqs) channels of x [n_tok][heads][d] by the tokens' positions (float64,
    no rounding): pairs (j, j + r/2), or (2j, 2j + 1) when interleaved; the other channels are copied."""
    x = np.array(x, dtype=np.float64, copy=True)
    h = len(freqs)
    for t, pos in enumerate(np.asarray(positions).tolist()):
        for j in range(h):
            i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + h)
            a = np.fmod(pos * freqs[j], 2 * np.pi)
            c, s = amp * np.cos(a), amp * np.sin(a)
            u, v = x[t, :, i0].copy(), x[t, :, i1].copy()
            x[t, :, i0], x[t, :, i1] = u * c - v * s, u * s + v * c
    return x
