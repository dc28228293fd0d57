"""CPU oracle for the quantised cache and the operators that read it (test
infrastructure only).

Plain numpy, float64 arithmetic.  It shares no code with the CUDA library.
The formats are the library's own definition (include/sige.h):

  * integers of 8 (4) bits: scale = float32(m / 127) (7) of the group's largest
    magnitude m, code = the exact quotient t / scale rounded to the nearest
    integer, ties to even;
  * e4m3: scale = 2^ceil(log2(m / 448)), code = t / scale rounded to the
    format, ties to even;
  * a scale below 2^-126 becomes 0 with codes 0; a group with an infinity or
    a NaN gets a NaN scale and codes 0.

A quotient in float64 decides every tie exactly: t and scale have 24-bit
significands, so 2 t and (2 k + 1) scale, both multiples of the scale's unit in
the last place when |t| >= scale / 2, differ by nothing or by more than a
float64 quotient's error.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle.attention import active_tokens, softmax_rows

QMAX = {"s8": 127.0, "s4": 7.0}
TINY = 2.0 ** -126


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """Float64 values of magnitude <= 448 rounded to e4m3 (3 mantissa bits,
    smallest normal 2^-6, spacing 2^-9 below), ties to even."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(np.where(v == 0, 1.0, v))            # |v| in [2^(e-1), 2^e)
    grid = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(v / grid) * grid


def e4m3_byte(v: float) -> int:
    """The byte of an e4m3 value (not -0)."""
    s, a = (128, -v) if v < 0 else (0, v)
    if a < 2.0 ** -6:
        return s | int(a * 2 ** 9)
    m, e = np.frexp(a)
    return s | (int(e - 1 + 7) << 3) | int((m * 2 - 1) * 8)


def quantise(t: np.ndarray, group: int, fmt: str):
    """(code values float64 [..., C], scales float32 [..., C / group]) of float32
    (or float64-held) values t [..., C]."""
    t = np.asarray(t, dtype=np.float64)
    g = t.reshape(*t.shape[:-1], -1, group)
    m = np.abs(g).max(-1)
    bad = ~np.isfinite(g).all(-1)
    m = np.where(bad, 0.0, m)
    if fmt == "e4m3":
        f, e = np.frexp(m)                                # 448 = 0.875 * 2^9
        s = np.where(m > 0, np.ldexp(1.0, np.maximum(e - 9 + (f > 0.875), -200)), 0.0)
    else:
        s = (m.astype(np.float32) / np.float32(QMAX[fmt])).astype(np.float64)
    s = np.where(s < TINY, 0.0, s)
    q = np.where((s > 0)[..., None] & ~bad[..., None], g, 0.0) / np.where(s > 0, s, 1.0)[..., None]
    q = e4m3_round(q) if fmt == "e4m3" else np.rint(q)
    s = np.where(bad, np.nan, s)
    return (q + 0.0).reshape(t.shape), s.astype(np.float32)


def stored(codes: np.ndarray, fmt: str) -> np.ndarray:
    """Code values as the bytes of a cache."""
    if fmt == "s8":
        return codes.astype(np.int8).view(np.uint8)
    if fmt == "e4m3":
        u, inv = np.unique(codes, return_inverse=True)
        return np.array([e4m3_byte(x) for x in u], dtype=np.uint8)[inv].reshape(codes.shape)
    n = codes.astype(np.int64) & 15
    return (n[..., 0::2] | (n[..., 1::2] << 4)).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """What code values stand for, float64."""
    s = np.asarray(scales, dtype=np.float64)
    return (codes.reshape(*s.shape, -1) * s[..., None]).reshape(codes.shape)


def qlinear(a, sa, w, sw, bias=None, residual=None) -> np.ndarray:
    """a [T, C], sa [T], w [O, C], sw [O] code values and scales -> float64 [T, O]."""
    acc = a.astype(np.int64) @ w.astype(np.int64).T
    y = acc.astype(np.float64) * np.asarray(sa, np.float64)[:, None] * np.asarray(sw, np.float64)[None]
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
    return y


def attention(q, k, v, heads: int, count=None):
    """q [T, D], k [L, D], v [L, Dv] float64 values; the first `count` keys.
    (o, |o|): the attention's rows and those over |v|, float64 [T, Dv]."""
    L = k.shape[0] if count is None else max(0, min(int(count), k.shape[0]))
    T, D = q.shape
    dv = v.shape[1]
    dh, dvh = D // heads, dv // heads
    o, oa = np.zeros((T, dv)), np.zeros((T, dv))
    for h in range(heads if L else 0):
        a, b = slice(h * dh, (h + 1) * dh), slice(h * dvh, (h + 1) * dvh)
        p = softmax_rows(q[:, a] @ k[:L, a].T / np.sqrt(dh))
        o[:, b] = p @ v[:L, b]
        oa[:, b] = p @ np.abs(v[:L, b])
    return o, oa


def tokens(idx, block: int, H: int, W: int) -> np.ndarray:
    """Active token ids of one item (every token when idx is None)."""
    return np.arange(H * W) if idx is None else active_tokens(idx, block, H, W)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to(torch.float64).cpu().numpy()
