"""Block-scaled e4m3 values and the gated linear over them (oracle; test infrastructure).

e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits, no infinities, code
0x7f = NaN; magnitudes 2^-9 .. 448. A matrix in 8 bits is its codes and one
float32 scale per block; the value of an element is code value * scale.

The quantiser is a float32 recipe (it fixes which code a tie gets), so it is
restated in float32 step by step; products over the values are fp64.
"""
from __future__ import annotations

import numpy as np

MAX = np.float32(448.0)
AMAX_FLOOR = np.float32(2.0 ** -100)


def code_values():
    """The 256 values of the codes, from the format's definition."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = np.nan if (c & 0x7F) == 0x7F else (-v if s else v)
    return out


def round_e4m3(v):
    """float64 values rounded to e4m3 (nearest, ties to the even code, saturating at 448)."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    _, e = np.frexp(np.where(a > 0, a, 1.0))          # a in [2^(e-1), 2^e)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))
    q = np.minimum(np.round(a / step) * step, 448.0)  # np.round: ties to even
    return np.copysign(q, v)


def _split(x, rows):
    M, K = x.shape
    for i in range(0, M, rows):
        for j in range(0, K, 128):
            yield i // rows, j // 128, (slice(i, min(i + rows, M)), slice(j, min(j + 128, K)))


def quantize(x, block_rows):
    """(e4m3 values [M,K] float64, scales float32) of a float32-exact x in blocks of block_rows x 128."""
    x = np.asarray(x, dtype=np.float32)
    M, K = x.shape
    vals = np.empty((M, K))
    scales = np.empty((-(-M // block_rows), -(-K // 128)), dtype=np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        for i, j, cut in _split(x, block_rows):
            amax = np.maximum(np.abs(x[cut]).max(), AMAX_FLOOR)   # np.maximum keeps a NaN
            scales[i, j] = np.float32(amax) / MAX
            vals[cut] = round_e4m3((x[cut] * (MAX / np.float32(amax))).astype(np.float64))
    return vals, scales


def values(codes, scales, block_rows):
    """Code values times block scales, in float64."""
    out = np.array(codes, dtype=np.float64)
    for i, j, cut in _split(out, block_rows):
        out[cut] *= float(scales[i, j])
    return out


def gated_linear_fp8(x, Wv, Ws, A, Bl, gate, scale):
    """y [M,N] = x^ W^^T + scale g (x A^T) Bl^T in float64; Wv: code values, x: bf16-exact floats.

    Returns (y, bound): bound is how far a computation with fp32 sums, bf16
    x A^T and a bf16 result may be from y. With u = 2^-23 an fp32 addition
    (whether it rounds or cuts off) changes a sum of n terms by at most
    n u sum|terms|: 128 terms in a block and one per block between them; the
    down-projection sums K terms and is rounded to bf16 (2^-8 of it), the
    up-projection sums r; the result is rounded to bf16 (2^-8 of it).
    """
    x = np.asarray(x, dtype=np.float64)
    xv, xs = quantize(x, 1)
    xh, wh = values(xv, xs, 1), values(Wv, Ws, 128)
    u = 2.0 ** -23
    K = x.shape[1]
    nkb = -(-K // 128)
    y = xh @ wh.T
    err = (128 + 4 * nkb) * u * (np.abs(xh) @ np.abs(wh).T)   # 4: the product of two scales and the fused add
    if A is not None:
        A, Bl = np.asarray(A, dtype=np.float64), np.asarray(Bl, dtype=np.float64)
        sg = float(scale) * np.asarray(gate, dtype=np.float64)[:, None]
        t = sg * (x @ A.T)
        dt = np.abs(sg) * K * u * (np.abs(x) @ np.abs(A).T) + 2.0 ** -8 * np.abs(t)
        y = y + t @ Bl.T
        err = err + dt @ np.abs(Bl).T + (A.shape[0] + 4) * u * (np.abs(t) @ np.abs(Bl).T)
    return y, 1.01 * err + 2.0 ** -8 * (np.abs(y) + err)


def gated_input_grad_fp8(dy, Wv, Ws, A, Bl, gate, scale):
    """dx [M,K] = dy^ W^ + scale g (dy Bl) A and its bound; Wv [N,K] code values, Ws as in the forward pass."""
    At = None if A is None else np.asarray(A).T
    Blt = None if Bl is None else np.asarray(Bl).T
    return gated_linear_fp8(dy, np.asarray(Wv).T, np.asarray(Ws).T, Blt, At, gate, scale)
