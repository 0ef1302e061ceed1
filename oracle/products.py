"""Oracle of the feed-forward products: the matrix product with bias, activation
and residual, the gated block, their backward passes, and 8-bit rows.

torch in float64 from the formulas of include/fq.h.  Next to each result stands
how far an implementation with FP32 sums may be from it, element by element:
  * a product of BF16 values is exact in FP32; a sum of K of them in any order is
    off by at most K 2^-24 times the sum of their magnitudes (twice that here,
    for adders that truncate);
  * FP32 evaluation of an activation from its formula: 16 units of 2^-24 of the
    argument's and the result's magnitude (the argument of exp is rounded too,
    which costs at most 0.6 |z| such units), its derivative 32 units;
  * the activations' slopes are at most 1.13;
  * a rounding to BF16 is off by at most 2^-8, to FP32 by 2^-24, of the value.
"""
from __future__ import annotations

import math

import torch

EPS32, EPS16 = 2.0 ** -24, 2.0 ** -8
SLOPE = 1.13
FLOOR = 1e-37                      # of what is rounded below the normal range
NONE, RELU, SILU, GELU = 0, 1, 2, 3


def act(z, kind, alpha=1.0):
    """The activation of z and its derivative."""
    if kind == RELU:
        return z.clamp_min(0.0), (z > 0).double()
    if kind == SILU:
        s = torch.sigmoid(alpha * z)
        return z * s, s * (1 + alpha * z * (1 - s))
    if kind == GELU:
        phi = 0.5 * (1 + torch.erf(z / math.sqrt(2)))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def act_close(z, kind, alpha=1.0):
    """(a(z), a'(z)) of SiLU or GELU and how far an FP32 evaluation of their formulas
    may be from either, relative to what they are: the side that falls to 0 keeps its
    precision.  In units of 2^-24, with exp2 and reciprocal to two of them:
      * exp(-v): v, its product with log2 e and that constant are rounded, 2.23 |v|,
        and 2; s = 1 / (1 + exp(-v)) takes the share 1 - s of that, and 3 more;
      * a = z s one more; a' = s + v s (1 - s), where 1 - s has the absolute error of s
        and a rounding, one product and one sum;
      * the normal distribution's smaller side q = exp(-z^2 / 2) t P(t) / 2: 1.12 z^2 + 2
        for the exponent; 3.8 for the polynomial's sums, 3 for t, which its slope makes at
        most 10, 0.4 for the fit; 2 products.  The other side is 1 - q;
      * a' = phi + z exp(-z^2 / 2) / sqrt(2 pi) from the same exponential.
    Where a reciprocal or exp2 that a result depends on is below the normal range, it may
    be lost whole (its border is moved by a factor of 2 for its own error); products below
    that range are rounded to 2^-150."""
    z = z.double()
    if kind == SILU:
        v = alpha * z
        s, c = torch.sigmoid(v), torch.sigmoid(-v)
        es = c * (2.3 * v.abs() + 2.1) + 3.1
        value, slope = z * s, s + v * s * c
        tv = (es + 1.1) * value.abs()
        td = es * s + v.abs() * s * (c * (es + 3.1) + s * es) + slope.abs()
        lost = torch.where(s < 2.0 ** -125, s, 0.0) * (1 + v.abs()) * (1 + z.abs())
    else:
        phi, q = (torch.special.erfc(side * z / math.sqrt(2)) / 2 for side in (-1, 1))
        pdf = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        eq = 1.15 * z * z + 19.0
        ephi = torch.where(z < 0, phi * eq, q * eq + 1.1)
        value, slope = z * phi, phi + z * pdf
        tv = z.abs() * ephi + 1.1 * value.abs()
        td = ephi + z.abs() * pdf * (1.15 * z * z + 7.0) + slope.abs()
        lost = torch.where(torch.exp(-0.5 * z * z) < 2.0 ** -125, q + z.abs() * pdf, 0.0) * (1 + z.abs())
    lost = lost + 2.0 ** -148 * (1 + z.abs())
    return value, slope, EPS32 * tv + lost, EPS32 * td + lost


def gate(z, g):
    """(a(g'), a'(g') or 0, u' + shift, 1 or 0) of z = [g, u]; g = (act, alpha, limit, shift)."""
    kind, alpha, limit, shift = g
    a, b = z.chunk(2, -1)
    v, dv = act(a.clamp_max(limit), kind, alpha)
    return v, torch.where(a > limit, 0.0, dv), b.clamp(-limit, limit) + shift, (b.abs() <= limit).double()


def segments(starts, rows, w):
    """(expert's weight, first row, end) of every segment."""
    if starts is None:
        return [(w, 0, rows)]
    return [(w[e], a, b) for e, (a, b) in enumerate(zip(starts, starts[1:]))]


def _half_step(v, dtype):
    return (EPS16 if dtype == torch.bfloat16 else EPS32) * v.abs() + FLOOR


def linear_fwd(x, w, bias, res, kind, starts=None, dtype=torch.bfloat16):
    """{"z", "y"} and {"z", "y"} of their bounds; rows of no segment are NaN."""
    x, w = x.double(), w.double()
    n = w.shape[-1]
    z, tz = (torch.full((x.shape[0], n), math.nan, dtype=torch.float64, device=x.device) for _ in range(2))
    for e, (we, a, b) in enumerate(segments(starts, x.shape[0], w)):
        be = torch.zeros(n, dtype=torch.float64, device=x.device) if bias is None else bias.double().view(-1, n)[e]
        z[a:b] = x[a:b] @ we + be
        tz[a:b] = 2 * (x.shape[1] + 2) * EPS32 * (x[a:b].abs() @ we.abs() + be.abs())
    y, _ = act(z, kind)
    ty = SLOPE * tz + (16 * EPS32 * (z.abs() + y.abs()) if kind else 0)
    if res is not None:
        y = y + res.double()
        ty = ty + 2 * EPS32 * (y.abs() + res.double().abs())
    return {"z": z, "y": y}, {"z": tz, "y": ty + _half_step(y.abs() + ty, dtype)}


def glu_fwd(x, w, bias, g, starts=None):
    v, t = linear_fwd(x, w, bias, None, NONE, starts)
    z, tz = v["z"], t["z"]
    a, _, up, _ = gate(z, g)
    tg, tu = tz.chunk(2, -1)
    ta = SLOPE * tg + 16 * EPS32 * (z.chunk(2, -1)[0].abs() + a.abs())
    tu = tu + 2 * EPS32 * (up.abs() + abs(g[3]))
    h = a * up
    th = ta * up.abs() + tu * a.abs() + ta * tu
    return {"z": z, "y": h}, {"z": tz, "y": th + _half_step(h.abs() + th, torch.bfloat16)}


def _bwd(d, td, x, w, starts, dw_dtype):
    """dx, dw, dbias of the gradient d before the activation, known to td."""
    x, w = x.double(), w.double()
    tz = td + _half_step(d.abs() + td, torch.bfloat16)
    v = {"dx": torch.full(x.shape, math.nan, dtype=torch.float64, device=x.device), "dw": torch.zeros_like(w),
         "dbias": torch.zeros(w.shape[:-2] + w.shape[-1:], dtype=torch.float64, device=x.device)}
    t = {k: torch.zeros_like(r) for k, r in v.items()}
    # what an output keeps of the roundings of dz and of its own sum
    for e, (we, a, b) in enumerate(segments(starts, x.shape[0], w)):
        at = (e,) if starts is not None else ()
        big = d[a:b].abs() + tz[a:b]
        v["dx"][a:b] = d[a:b] @ we.T
        t["dx"][a:b] = tz[a:b] @ we.abs().T + 2 * (w.shape[-1] + 2) * EPS32 * (big @ we.abs().T)
        v["dw"][at] = x[a:b].T @ d[a:b]
        t["dw"][at] = x[a:b].abs().T @ tz[a:b] + 2 * (b - a + 2) * EPS32 * (x[a:b].abs().T @ big)
        v["dbias"][at] = d[a:b].sum(0)
        t["dbias"][at] = td[a:b].sum(0) + 2 * (b - a + 2) * EPS32 * d[a:b].abs().sum(0)
    for k, dtype in (("dx", torch.bfloat16), ("dw", dw_dtype), ("dbias", torch.float32)):
        t[k] = t[k] + _half_step(v[k].abs() + t[k], dtype)
    return v, t


def linear_bwd(dy, x, w, pre, kind, starts=None, dw_dtype=torch.bfloat16):
    d, td = dy.double(), torch.zeros_like(dy.double())
    if kind == NONE:
        # dz is dy itself: no rounding of it
        v, t = _bwd(d, td, x, w, starts, dw_dtype)
        _, exact = _bwd_exact(d, x, w, starts, dw_dtype)
        return v, exact
    td = 32 * EPS32 * d.abs() if kind != RELU else td
    return _bwd(d * act(pre.double(), kind)[1], td, x, w, starts, dw_dtype)


def _bwd_exact(d, x, w, starts, dw_dtype):
    x, w = x.double(), w.double()
    v, t = {}, {"dx": torch.zeros_like(x), "dw": torch.zeros_like(w),
                "dbias": torch.zeros(w.shape[:-2] + w.shape[-1:], dtype=torch.float64, device=x.device)}
    for e, (we, a, b) in enumerate(segments(starts, x.shape[0], w)):
        at = (e,) if starts is not None else ()
        big = d[a:b].abs()
        for k, value, size, n, dtype in (
                ("dx", d[a:b] @ we.T, big @ we.abs().T, w.shape[-1], torch.bfloat16),
                ("dw", x[a:b].T @ d[a:b], x[a:b].abs().T @ big, b - a, dw_dtype),
                ("dbias", d[a:b].sum(0), big.sum(0), b - a, torch.float32)):
            bound = 2 * (n + 2) * EPS32 * size
            bound = bound + _half_step(value.abs() + bound, dtype)
            t[k][slice(a, b) if k == "dx" else at] = bound
    return v, t


def glu_bwd(dh, x, w, pre, g, starts=None, dw_dtype=torch.bfloat16):
    z, d = pre.double(), dh.double()
    a, da, up, inside = gate(z, g)
    grad = torch.cat((d * up * da, d * a * inside), -1)
    ta = 16 * EPS32 * (z.chunk(2, -1)[0].clamp_max(g[2]).abs() + a.abs())
    td = torch.cat((32 * EPS32 * d.abs() * (up.abs() + abs(g[3])), d.abs() * (ta + 2 * EPS32 * a.abs())), -1)
    v, t = _bwd(grad, td, x, w, starts, dw_dtype)
    v["h"] = a * up
    th = ta * up.abs() + 2 * EPS32 * (up.abs() + abs(g[3])) * a.abs()
    t["h"] = th + _half_step(v["h"].abs() + th, torch.bfloat16)
    return v, t


# ---------------------------------------------------------------------------
# 8-bit rows
# ---------------------------------------------------------------------------

def pow2(e):
    """2^e of whole numbers e in -200 .. 200, exactly (a device's pow may not be)."""
    table = torch.tensor([2.0 ** i for i in range(-200, 201)], dtype=torch.float64, device=e.device)
    return table[e.long() + 200]


def e4m3_values(device="cpu"):
    """Values of codes 0 .. 126 of E4M3."""
    c = torch.arange(127, device=device)
    e, m = c // 8, (c % 8).double()
    return torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * pow2(e - 7))


def encode_mx(x):
    """(codes, E8M0 codes) of the rows x, from the definition in float64."""
    rows, cols = x.shape
    b = x.double().reshape(rows, cols // 32, 32)
    top = b.abs().amax(2)
    bad = ~torch.isfinite(top)
    e = torch.ceil(torch.log2(torch.where((top == 0) | bad, 448.0 * 2.0 ** -127, top) / 448.0)).clamp(-127, 127)
    codes = _nearest(b / pow2(e)[:, :, None])
    codes = torch.where(bad[:, :, None], 0x7F, codes)
    return codes.reshape(rows, cols).to(torch.uint8), torch.where(bad, 255.0, e + 127).to(torch.uint8)


def encode_row(x):
    """(codes, FP32 scales): products of FP32 numbers rounded to FP32."""
    top = x.float().abs().amax(1)
    bad = ~torch.isfinite(top)
    seventh = torch.tensor(1.0 / 448.0, dtype=torch.float64).float().double()
    s = (torch.where(bad, 1.0, top).double() * seventh.to(x.device)).float().clamp_min(2.0 ** -126)
    inv = (1.0 / s.double()).float()
    a = (torch.where(bad[:, None], 0.0, x.float()).double() * inv.double()[:, None]).float().clamp(-448, 448)
    codes = torch.where(bad[:, None], 0x7F, _nearest(a.double()))
    return codes.to(torch.uint8), torch.where(bad, math.nan, s)


def _nearest(a):
    """E4M3 codes of |a| <= 448, to nearest, ties to the even code, the sign kept."""
    v = e4m3_values(a.device)
    m = a.abs()
    k = torch.searchsorted(v, m.contiguous(), right=True) - 1
    up = (k + 1).clamp_max(126)
    mid = (v[k] + v[up]) / 2
    k = torch.where((m > mid) | ((m == mid) & (k % 2 == 1)), up, k)
    return k + torch.where(torch.signbit(a), 128, 0)


def decode(codes, scales, mx):
    """The values in float64, before their rounding to BF16."""
    c = codes.long()
    v = torch.cat((e4m3_values(codes.device), torch.tensor([math.nan], dtype=torch.float64, device=codes.device)))[c & 127]
    v = torch.where(c >= 128, -v, v)
    if not mx:
        return v * scales.double()[:, None]
    s = torch.where(scales == 255, math.nan, pow2(scales.long() - 127))
    return v * s.repeat_interleave(32, 1)
