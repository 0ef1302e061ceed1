"""Oracle of the operators around the quantized linears: residual addition
with root-mean-square norm and its backward, expert sorting, AdamW.

numpy in float64 from the formulas of include/fq.h, with the roundings that
the definitions name (BF16, E4M3, E5M2, FP32 scales) done explicitly.  Loops
where the definition is a loop; for small inputs.
"""
from __future__ import annotations

import numpy as np

import oracle

TINY = 2.0 ** -126


# ---------------------------------------------------------------------------
# 8-bit floats (OCP OFP8 v1.0)
# ---------------------------------------------------------------------------

def float8_values(mant: int) -> np.ndarray:
    """Values of the non-negative codes 0 .. 127 of E4M3 (mant = 3) or E5M2
    (mant = 2); NaN / infinity where the format has them."""
    bias = {3: 7, 2: 15}[mant]
    v = np.empty(128)
    for c in range(128):
        e, m = c >> mant, c & ((1 << mant) - 1)
        v[c] = (m * 2.0 ** (1 - bias - mant) if e == 0
                else (1 + m / (1 << mant)) * 2.0 ** (e - bias))
    if mant == 3:
        v[127] = np.nan
    else:
        v[124], v[125:] = np.inf, np.nan
    return v


E4M3, E5M2 = float8_values(3), float8_values(2)
E4M3_MAX, E5M2_MAX = 448.0, 57344.0


def float8_decode(codes: np.ndarray, table: np.ndarray) -> np.ndarray:
    v = table[codes & 0x7F]
    return np.where(codes & 0x80, -v, v)


def float8_sr(a: np.ndarray, r16: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Codes of 0 <= a <= largest: up where r16 < floor(2^16 * fraction)."""
    finite = table[np.isfinite(table)]
    k = np.searchsorted(finite, a, side="right") - 1
    above = np.minimum(k + 1, finite.size - 1)
    gap = np.where(above > k, finite[above] - finite[k], 1.0)
    t = np.floor((a - finite[k]) / gap * 65536)
    return (k + (r16 < t)).astype(np.uint8)


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

def bf16_round(x: np.ndarray) -> np.ndarray:
    """float32 -> nearest BF16 value (as float32), ties to even; infinities and
    NaN stay what they are."""
    x = np.ascontiguousarray(x, np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(x), r, x)


def residual(x: np.ndarray, res: np.ndarray, bf16: bool) -> np.ndarray:
    h = (x.astype(np.float32) + res.astype(np.float32)).astype(np.float32)
    return bf16_round(h) if bf16 else h


def rmsnorm(h: np.ndarray, gamma: np.ndarray, eps: float):
    """(n, rstd) in float64."""
    h = h.astype(np.float64)
    r = 1 / np.sqrt((h * h).mean(1) + float(np.float32(eps)))
    return h * r[:, None] * gamma.astype(np.float64), r


def rmsnorm_bwd(dy, h, gamma, rstd, dres=None):
    """(dh, dgamma) in float64."""
    dy, h, gamma, r = (np.asarray(t, np.float64) for t in (dy, h, gamma, rstd))
    xh = h * r[:, None]
    g = dy * gamma
    dh = r[:, None] * (g - xh * (g * xh).mean(1, keepdims=True))
    if dres is not None:
        dh = dh + dres
    return dh, (dy * xh).sum(0)


def mx8_scale_code(amax: np.ndarray) -> np.ndarray:
    """E8M0 code of the smallest 2^e with amax <= 448 * 2^e."""
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(np.asarray(amax, np.float64) / 448))
    return (np.clip(e, -127, 127) + 127).astype(np.int64)


# ---------------------------------------------------------------------------
# expert sorting
# ---------------------------------------------------------------------------

def moe_sort(ids: np.ndarray, experts: int, align: int, rows: int):
    flat = ids.reshape(-1)
    pos, src = np.full(flat.size, -1, np.int32), np.full(rows, -1, np.int32)
    offsets = np.zeros(experts + 1, np.int32)
    at = 0
    for e in range(experts):
        offsets[e] = at
        mine = np.flatnonzero(flat == e)
        pos[mine] = at + np.arange(mine.size)
        src[at: at + mine.size] = mine
        at += -(-mine.size // align) * align
    offsets[experts] = at
    return offsets, pos.reshape(ids.shape), src


def moe_rows_of(x: np.ndarray, src: np.ndarray, k: int) -> np.ndarray:
    y = np.zeros((src.size, x.shape[1]), x.dtype)
    y[src >= 0] = x[src[src >= 0] // k]
    return y


def moe_combine(y: np.ndarray, pos: np.ndarray, weights=None) -> np.ndarray:
    out = np.zeros((pos.shape[0], y.shape[1]))
    for t in range(pos.shape[0]):
        for j in range(pos.shape[1]):
            if pos[t, j] >= 0:
                out[t] += (1.0 if weights is None else float(weights[t, j])) * y[pos[t, j]].astype(np.float64)
    return out


def moe_combine_bwd(dout, y, pos, weights):
    dy = np.zeros(y.shape)
    dw = np.zeros(pos.shape)
    for t in range(pos.shape[0]):
        for j in range(pos.shape[1]):
            if pos[t, j] >= 0:
                dy[pos[t, j]] = float(weights[t, j]) * dout[t].astype(np.float64)
                dw[t, j] = dout[t].astype(np.float64) @ y[pos[t, j]].astype(np.float64)
    return dy, dw


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

def adamw(w, g, m, v, *, lr, step, beta1, beta2, eps, weight_decay, scale=1.0):
    """(w, m, v) in float64."""
    w, g, m, v = (np.asarray(t, np.float64) for t in (w, g, m, v))
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    w = w * (1 - lr * weight_decay)
    return w - lr / (1 - beta1 ** step) * m / (np.sqrt(v) / np.sqrt(1 - beta2 ** step) + eps), m, v


def state_draws(n: int, tensor: int, step: int, seed: int):
    """(r16 of m, r16 of v) for the elements 0 .. n - 1 of a tensor."""
    words = np.empty((-(-n // 4), 4), np.uint32)
    for q in range(words.shape[0]):
        words[q] = oracle.philox4x32_10([q & 0xFFFFFFFF, q >> 32, tensor, step],
                                        [seed & 0xFFFFFFFF, seed >> 32])
    words = words.reshape(-1)[:n]
    return (words & 0xFFFF).astype(np.int64), (words >> 16).astype(np.int64)


def quantize_state(x: np.ndarray, r16: np.ndarray, largest: float, table: np.ndarray,
                   keep_positive: bool):
    """(codes, scales) of FP32 moments x in blocks of 128."""
    x = np.asarray(x, np.float32)
    n = x.size
    codes, scales = np.zeros(n, np.uint8), np.zeros(-(-n // 128), np.float32)
    for b in range(scales.size):
        s = slice(128 * b, min(n, 128 * b + 128))
        xb = x[s]
        ok = np.isfinite(xb)
        amax = np.abs(xb[ok]).max() if ok.any() else np.float32(0)
        scale = max(np.float32(amax * np.float32(1 / largest)), np.float32(TINY))
        inv = np.float32(1) / scale
        a = np.minimum(np.abs(np.where(ok, xb, 0)) * inv, np.float32(largest)).astype(np.float32)
        c = float8_sr(a.astype(np.float64), r16[s], table)
        if keep_positive:
            c = np.where(xb > 0, np.maximum(c, 1), c)
        c = np.where(ok, c, 0x7F)
        codes[s] = c | np.where(np.signbit(xb), 0x80, 0) if not keep_positive else c
        scales[b] = scale
    return codes, scales
