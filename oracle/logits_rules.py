"""Token records and logits rules (oracle; test infrastructure).

One record per sequence: which ids its prompt holds and how often it emitted
each (a 16-bit word per id: bit 15 and bits 0..14). Rules on a row of logits,
with n(v) the emitted count of id v plus its occurrences on the row's path:
repetition divides positive and multiplies other logits of ids seen anywhere,
frequency and presence subtract per emission and once, biases add, and ids the
mask forbids become -inf. fp64 from exactly widened inputs.
"""
from __future__ import annotations

import numpy as np


def counts_add(counts, tokens, lens=None, slots=None, prompt=False):
    """counts [S,V] uint16 after the call, and whether an id or slot was out of range."""
    c = np.array(counts, dtype=np.uint16)
    bad = False
    for b in range(tokens.shape[0]):
        n = tokens.shape[1] if lens is None else min(int(lens[b]), tokens.shape[1])
        for t in tokens[b, :max(n, 0)]:
            s = b if slots is None else int(slots[b])
            if t == -1:
                continue
            if not (0 <= t < c.shape[1] and 0 <= s < c.shape[0]):
                bad = True
                continue
            w = int(c[s, t])
            c[s, t] = (w | 0x8000) if prompt else (w & 0x8000) | min((w & 0x7FFF) + 1, 0x7FFF)
    return c, bad


def process(logits, counts=None, slots=None, path=None, repetition=None, frequency=None,
            presence=None, bias_ids=None, bias=None, mask=None):
    """out [B,R,V] float64. path [B,P] (row j follows the first j ids) or [B,R,P]."""
    z = np.array(logits, dtype=np.float64)
    B, R, V = z.shape
    f32 = lambda a, b, d: d if a is None else float(np.float32(a[b]))   # noqa: E731
    for b in range(B):
        s = b if slots is None else int(slots[b])
        rec = np.zeros(V, np.uint16) if counts is None or not 0 <= s < counts.shape[0] else counts[s]
        rho, freq, pres = f32(repetition, b, 1.0), f32(frequency, b, 0.0), f32(presence, b, 0.0)
        for j in range(R):
            n = (rec & 0x7FFF).astype(np.int64)
            ids = [] if path is None else path[b, j] if path.ndim == 3 else path[b, :j]
            for t in ids:
                if 0 <= t < V:
                    n[t] += 1
            row = z[b, j]
            with np.errstate(invalid="ignore"):
                held = (n > 0) | (rec >= 0x8000)
                row = np.where(held, np.where(row > 0, row / rho, row * rho), row)
                row = row - freq * n - pres * (n > 0)
            if bias_ids is not None:
                for t, a in zip(bias_ids[b], bias[b]):
                    if 0 <= t < V:
                        row[t] += float(np.float32(a))
            if mask is not None:
                on = np.unpackbits(np.ascontiguousarray(mask[b, j]).view(np.uint8), bitorder="little")[:V]
                row = np.where(on != 0, row, -np.inf)
            z[b, j] = row
    return z
