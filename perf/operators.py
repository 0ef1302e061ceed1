"""The operators around the quantized linears of a training step, as cases to
measure: residual addition with root-mean-square norm (BF16 or 8-bit output)
and its backward, tokens sorted by expert and back with their weights and the
gradient of that, and AdamW over many tensors with FP32 or 8-bit states.

`own` chooses between the library's kernels and the plain form (elementary
torch operations in FP32).  Values held in 8 bits are returned as torch's
8-bit float types over the same bytes: codes as float8_e4m3fn / float8_e5m2,
power-of-two scales as float8_e8m0fnu.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-5
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP, GRAD_SCALE = 1e-4, 0.9, 0.95, 1e-8, 0.1, 12, 0.5
STATE_BLOCK = 128
TINY = 2.0 ** -126

F8 = {"none": 0, "mx": 1, "row": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token being decoded: stream and norm for an 8-bit product, latency only
        {"name": "norm 1x2880 8-bit", "op": "norm_fwd", "rows": 1, "cols": 2880, "stream": "bf16", "f8": "mx", "y": False},
        # a training step's activations: stream, fake-quantized output and its 8-bit codes
        {"name": "norm 16384x4096 8-bit", "op": "norm_fwd", "rows": 16384, "cols": 4096, "stream": "bf16", "f8": "mx", "y": True},
        # a ragged batch over an odd width, FP32 residual stream, BF16 output
        {"name": "norm 1777x2881 fp32", "op": "norm_fwd", "rows": 1777, "cols": 2881, "stream": "f32", "f8": "none", "y": True},
        # the training step's backward at the linears' size
        {"name": "norm bwd 8192x2880", "op": "norm_bwd", "rows": 8192, "cols": 2880, "stream": "bf16"},
        # backward of a short ragged batch with an FP32 stream
        {"name": "norm bwd 333x1000 fp32", "op": "norm_bwd", "rows": 333, "cols": 1000, "stream": "f32"},
        # one token through four of 32 experts
        {"name": "moe 1 token", "op": "moe_fwd", "tokens": 1, "k": 4, "experts": 32, "cols": 2880, "align": 1, "f8": "none", "masked": 0.0},
        # a training batch, rows kept in 8 bits until they are sorted, segments padded for the backward's products
        {"name": "moe 8192 tokens 8-bit", "op": "moe_fwd", "tokens": 8192, "k": 4, "experts": 32, "cols": 2880, "align": 128, "f8": "mx", "masked": 0.0},
        # a ragged batch with padding tokens that no expert takes, many experts
        {"name": "moe 1021 tokens masked", "op": "moe_fwd", "tokens": 1021, "k": 8, "experts": 128, "cols": 1000, "align": 64, "f8": "none", "masked": 0.2},
        # the training batch's backward: rows' and weights' gradients, then the tokens'
        {"name": "moe bwd 8192 tokens", "op": "moe_bwd", "tokens": 8192, "k": 4, "experts": 32, "cols": 2880, "align": 128, "masked": 0.0},
        # a handful of norm gains and router rows
        {"name": "adamw 12 small", "op": "adamw", "count": 12, "size": 2880, "spread": 0.0, "states": "f32", "grads": "f32"},
        # expert weights with FP32 states
        {"name": "adamw 6 experts fp32", "op": "adamw", "count": 6, "size": 2880 * 5760, "spread": 0.0, "states": "f32", "grads": "bf16"},
        # many tensors of very different lengths with 8-bit states
        {"name": "adamw 200 ragged 8-bit", "op": "adamw", "count": 200, "size": 600000, "spread": 3.0, "states": "f8", "grads": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_fwd", "norm_bwd", "moe_fwd", "moe_bwd", "adamw"])
    if op in ("norm_fwd", "norm_bwd"):
        cols = _log(rng, 64, 16384)
        rows = min(_log(rng, 1, 32768), (1 << 26) // cols)
        stream = rng.choice(["bf16", "f32", "none"])
        if op == "norm_bwd":
            return {"op": op, "rows": min(rows, (1 << 25) // cols), "cols": cols, "stream": stream}
        f8 = rng.choice(["none", "mx", "row"])
        cols = cols if f8 == "none" else max(32, cols // 32 * 32)
        return {"op": op, "rows": rows, "cols": cols, "stream": stream, "f8": f8, "y": f8 == "none" or rng.random() < 0.5}
    if op in ("moe_fwd", "moe_bwd"):
        experts = _log(rng, 4, 256)
        k = rng.choice([1, 2, 4, 6, 8])
        k = min(k, experts)
        f8 = rng.choice(["none", "mx", "row"]) if op == "moe_fwd" else "none"
        cols = _log(rng, 64, 8192)
        cols = max(8, cols // 8 * 8) if f8 == "none" else max(32, cols // 32 * 32)
        tokens = max(1, min(_log(rng, 1, 16384), (8192 * 4 * 2880 // 2) // (k * cols)))
        c = {"op": op, "tokens": tokens, "k": k, "experts": experts, "cols": cols, "align": rng.choice([1, 16, 64, 128]),
             "masked": rng.choice([0.0, 0.0, 0.1, 0.5])}
        return dict(c, f8=f8) if op == "moe_fwd" else c
    states = rng.choice(["f32", "f8"])
    count = _log(rng, 1, 256)
    size = min(_log(rng, 1, 1 << 24), (1 << 25) // count)
    return {"op": op, "count": count, "size": max(1, size), "spread": rng.choice([0.0, 0.5, 2.0]), "states": states,
            "grads": rng.choice(["bf16", "f32"])}


def _capacity(c):
    n = c["tokens"] * c["k"]
    return (n + min(c["experts"], n) * (c["align"] - 1)) // c["align"] * c["align"]


def _sizes(c):
    """Lengths of the tensors: `size` times factors from 2^-spread to 2^spread,
    in an order that is the same for every seed."""
    n = c["count"]
    f = [2.0 ** (c["spread"] * ((i * 7919) % n * 2 / max(1, n - 1) - 1)) for i in range(n)]
    return [max(1, int(c["size"] * x)) for x in f]


def work(c):
    if c["op"] in ("norm_fwd", "norm_bwd"):
        n, s = c["rows"] * c["cols"], {"bf16": 2, "f32": 4, "none": 0}[c["stream"]]
        if c["op"] == "norm_fwd":
            per = 2 + 2 * s + (2 if c["y"] else 0)
            per += {"none": 0, "mx": 1 + 1 / 32, "row": 1 + 4 / c["cols"]}[c["f8"]]
            return {"bytes": n * per + 4 * c["rows"] + 4 * c["cols"], "flops": 5 * n}
        per = 2 + (3 * s + (2 if s == 4 else 0) if s else 4)
        return {"bytes": n * per + 4 * c["rows"] + 8 * c["cols"], "flops": 10 * n}
    if c["op"] in ("moe_fwd", "moe_bwd"):
        n, h, cap = c["tokens"] * c["k"], c["cols"], _capacity(c)
        live = n * (1 - c["masked"])
        if c["op"] == "moe_fwd":
            x = c["tokens"] * {"none": 2 * h, "mx": h + h / 32, "row": h + 4}[c["f8"]]
            return {"bytes": x + cap * h * 2 + live * h * 2 + c["tokens"] * h * 2 + 12 * n + 4 * cap + 4 * c["experts"],
                    "flops": 2 * live * h}
        # combine's backward, then dispatch's
        return {"bytes": c["tokens"] * h * 2 + live * h * 2 + cap * h * 2 + live * h * 2 + c["tokens"] * h * 2 + 12 * n + 4 * cap,
                "flops": 4 * live * h}
    n = sum(_sizes(c))
    g = 2 if c["grads"] == "bf16" else 4
    s = 16 if c["states"] == "f32" else 4 + 16 / STATE_BLOCK
    return {"bytes": n * (8 + 2 + g + s), "flops": 14 * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, sigma, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV) * sigma).to(dtype)


def _e8m0_codes(amax):
    """Biased exponent of the smallest power of two 2^e with amax <= 448 * 2^e."""
    u = amax.view(torch.int32)
    e = (u >> 23) - 8 + ((u & 0x7FFFFF) > 0x600000).int()
    return e.clamp(0, 254).to(torch.uint8)


def _pow2(codes):
    return torch.ldexp(torch.ones((), device=codes.device), codes.int() - 127)


def _norm_inputs(c, g):
    rows, cols = c["rows"], c["cols"]
    gain = 1 + 0.1 * torch.randn(cols, generator=g, device=DEV)
    s = {"gain": gain}
    channels = torch.randperm(cols, generator=g, device=DEV)[: max(1, cols // 512)]
    x = _normal(g, (rows, cols), 1.0)
    stream = None
    if c["stream"] != "none":
        stream = torch.randn((rows, cols), generator=g, device=DEV) * 2
        stream[:, channels] *= 20                      # the few channels with large values
        stream = stream if c["stream"] == "f32" else stream.to(torch.bfloat16)
    if c["op"] == "norm_fwd":
        return dict(s, x=x, res=stream)
    h = x if stream is None else (x.float() + stream.float()).to(stream.dtype)
    s["h"] = h
    s["rstd"] = torch.rsqrt(h.float().square().mean(1) + EPS)
    s["dy"] = _normal(g, (rows, cols), 1e-3)
    s["dres"] = None if stream is None else _normal(g, (rows, cols), 1e-3, h.dtype)
    return s


def _moe_inputs(c, g):
    t, k, n, h = c["tokens"], c["k"], c["experts"], c["cols"]
    # experts are not equally liked: their logits have a bias of their own
    logits = torch.randn((t, n), generator=g, device=DEV) + 0.5 * torch.randn(n, generator=g, device=DEV)
    top, ids = logits.topk(k, dim=1)
    ids = ids.to(torch.int32)
    if c["masked"]:
        ids[torch.rand(t, generator=g, device=DEV) < c["masked"]] = -1       # padding tokens
    s = {"ids": ids, "weights": torch.softmax(top, 1), "y": _normal(g, (_capacity(c), h), 1.0)}
    if c["op"] == "moe_bwd":
        s["dout"] = _normal(g, (t, h), 1e-3)
        s["dx_rows"] = _normal(g, (_capacity(c), h), 1e-3)      # what the experts' linears give back
        s["offsets"], s["pos"], s["src"] = _sort(c, ids)
        return s
    x = _normal(g, (t, h), 1.0)
    if c["f8"] == "none":
        return dict(s, x=x, scales=None)
    v = x.float()
    if c["f8"] == "mx":
        scales = _e8m0_codes(v.view(t, h // 32, 32).abs().amax(2))
        q = v / _pow2(scales).repeat_interleave(32, 1)
    else:
        scales = (v.abs().amax(1) / 448).clamp_min(TINY)
        q = (v * (1 / scales)[:, None]).clamp(-448, 448)
    return dict(s, x=q.to(torch.float8_e4m3fn).view(torch.uint8), scales=scales)


def _adamw_inputs(c, g):
    """All tensors in one buffer each for w, g, m, v (every tensor starts at a
    multiple of the states' block), and where each begins."""
    sizes = _sizes(c)
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += (n + STATE_BLOCK - 1) // STATE_BLOCK * STATE_BLOCK
    live = torch.ones(at, device=DEV)
    for a, n in zip(starts, sizes):
        live[a + n: a + (n + STATE_BLOCK - 1) // STATE_BLOCK * STATE_BLOCK] = 0
    s = {"sizes": sizes, "starts": starts}
    s["w"] = torch.randn(at, generator=g, device=DEV) * 0.02 * live
    s["w16"] = s["w"].to(torch.bfloat16)
    # gradients of one tensor differ in size from row to row
    rough = torch.exp(torch.randn(at // STATE_BLOCK, generator=g, device=DEV)).repeat_interleave(STATE_BLOCK) * live
    grad = torch.randn(at, generator=g, device=DEV) * 1e-3 * rough
    s["g"] = grad if c["grads"] == "f32" else grad.to(torch.bfloat16)
    s["scale"] = torch.full((1,), GRAD_SCALE, device=DEV)
    m = torch.randn(at, generator=g, device=DEV) * 3e-4 * rough
    v = (torch.randn(at, generator=g, device=DEV) * 1e-3 * rough).square() * 0.3
    if c["states"] == "f32":
        return dict(s, m=m, v=v, seed=0)
    ms = (m.view(-1, STATE_BLOCK).abs().amax(1) / 448).clamp_min(TINY)
    vs = (v.view(-1, STATE_BLOCK).amax(1) / 57344).clamp_min(TINY)
    m = (m.view(-1, STATE_BLOCK) / ms[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(-1)
    v = (v.view(-1, STATE_BLOCK) / vs[:, None]).clamp(0, 57344).to(torch.float8_e5m2).view(-1)
    return dict(s, m=m.view(torch.uint8), v=v.view(torch.uint8), ms=ms, vs=vs,
                seed=int(torch.randint(1 << 40, (1,), generator=g, device=DEV)))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = (_norm_inputs if op.startswith("norm") else _moe_inputs if op.startswith("moe") else _adamw_inputs)(case, g)
    s["case"] = case
    if own:
        s["out"] = _buffers(case, s)
    return s


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _buffers(c, s):
    """What a program that calls the library keeps between steps: its output
    buffers, its workspaces and the list of tensors of its optimizer."""
    import fp4_block_quantization_fq_amd as fq
    new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    if c["op"] == "norm_fwd":
        rows, cols = c["rows"], c["cols"]
        o = {"h": None if s["res"] is None else torch.empty_like(s["res"]), "rstd": new(rows, f32)}
        o["y"] = new((rows, cols), bf) if c["y"] else None
        o["codes"] = new((rows, cols), u8) if c["f8"] != "none" else None
        o["scales"] = {"none": None, "mx": new((rows, cols // 32), u8), "row": new(rows, f32)}[c["f8"]]
        return o
    if c["op"] == "norm_bwd":
        h = s["h"]
        ws = fq.rmsnorm_bwd_workspace(c["rows"], c["cols"], DEV)
        return {"dh": torch.empty_like(h), "dx": new(h.shape, bf) if h.dtype == f32 else None, "dgamma": new(c["cols"], f32), "ws": ws}
    if c["op"].startswith("moe"):
        t, k, h = c["tokens"], c["k"], c["cols"]
        rows = fq.moe_rows(t, k, c["experts"], c["align"])
        o = {"sorted": fq.MoeSorted(new(c["experts"] + 1, i32), new((t, k), i32), new(rows, i32)),
             "ws": fq.moe_sort_workspace(t, k, c["experts"], DEV),
             "rows": new((rows, h), bf), "out": new((t, h), bf), "dw": new((t, k), f32)}
        if c["op"] == "moe_bwd":
            o["sorted"] = fq.MoeSorted(s["offsets"], s["pos"], s["src"])
        return o
    tensors = []
    for a, n in zip(s["starts"], s["sizes"]):
        b = (a // STATE_BLOCK, (a + n + STATE_BLOCK - 1) // STATE_BLOCK)
        scales = {} if c["states"] == "f32" else {"m_scale": s["ms"][b[0]:b[1]], "v_scale": s["vs"][b[0]:b[1]]}
        tensors.append(fq.AdamWTensor(w=s["w"][a:a + n], g=s["g"][a:a + n], m=s["m"][a:a + n], v=s["v"][a:a + n],
                                      w_bf16=s["w16"][a:a + n], weight_decay=DECAY, **scales))
    return {"plan": fq.adamw_plan(tensors)}


def _run_own(s):
    import fp4_block_quantization_fq_amd as fq
    c, o = s["case"], s["out"]
    f8 = (fq.FQ_F8_NONE, fq.FQ_F8_MX, fq.FQ_F8_ROW)[F8[c.get("f8", "none")]]
    if c["op"] == "norm_fwd":
        fq.fq_rmsnorm_fwd(s["x"], s["gain"], EPS, res=s["res"], f8=f8, h=o["h"], y=o["y"], codes=o["codes"],
                          scales=o["scales"], rstd=o["rstd"])
        return _norm_out(c, o["h"], o["y"], o["codes"], o["scales"], o["rstd"])
    if c["op"] == "norm_bwd":
        fq.fq_rmsnorm_bwd(s["dy"], s["h"], s["gain"], s["rstd"], dres=s["dres"], dh=o["dh"], dx=o["dx"],
                          dgamma=o["dgamma"], ws=o["ws"])
        return {"dh": o["dh"], "dx": o["dx"], "dgamma": o["dgamma"]}
    if c["op"] == "moe_fwd":
        q = fq.fq_moe_sort(s["ids"], c["experts"], c["align"], out=o["sorted"], ws=o["ws"])
        fq.fq_moe_dispatch(s["x"], q, f8=f8, scales=s["scales"], y=o["rows"])
        fq.fq_moe_combine(s["y"], q, s["weights"], out=o["out"])
        return {"offsets": q.offsets, "pos": q.pos, "src": q.src, "rows": o["rows"], "out": o["out"]}
    if c["op"] == "moe_bwd":
        fq.fq_moe_combine_bwd(s["dout"], s["y"], o["sorted"], s["weights"], dy=o["rows"], dweights=o["dw"])
        fq.fq_moe_combine(s["dx_rows"], o["sorted"], None, out=o["out"])
        return {"dy": o["rows"], "dw": o["dw"], "dx": o["out"]}
    fq.fq_adamw_step(o["plan"], lr=LR, step=STEP, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, grad_scale=s["scale"],
                     seed=s["seed"])
    return _adamw_out(s)


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

def _norm_out(c, h, y, codes, scales, rstd):
    o = {"h": h, "y": y, "rstd": rstd}
    if codes is not None:
        o["codes"] = codes.view(torch.float8_e4m3fn)
        o["scales"] = scales.view(torch.float8_e8m0fnu) if c["f8"] == "mx" else scales
    return o


def _norm_fwd(s):
    c = s["case"]
    h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["res"].dtype)
    v = h.float()
    rstd = 1 / torch.sqrt(v.square().mean(1) + EPS)
    n = v * rstd[:, None] * s["gain"]
    codes = scales = None
    y = n.to(torch.bfloat16)
    rows, cols = n.shape
    if c["f8"] == "mx":
        b = n.view(rows, cols // 32, 32)
        scales = _e8m0_codes(b.abs().amax(2))
        p = _pow2(scales)[:, :, None]
        q = (b / p).to(torch.float8_e4m3fn)
        y = (q.float() * p).view(rows, cols).to(torch.bfloat16)
        codes = q.view(rows, cols).view(torch.uint8)
    elif c["f8"] == "row":
        scales = (n.abs().amax(1) / 448).clamp_min(TINY)
        q = (n * (1 / scales)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        y = (q.float() * scales[:, None]).to(torch.bfloat16)
        codes = q.view(torch.uint8)
    return _norm_out(c, None if s["res"] is None else h, y if c["y"] else None, codes, scales, rstd)


def _norm_bwd(s):
    xh = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["gain"]
    dh = s["rstd"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dh = dh + s["dres"].float()
    dgamma = (dy * xh).sum(0)
    wide = s["h"].dtype == torch.float32
    return {"dh": dh.to(s["h"].dtype), "dx": dh.to(torch.bfloat16) if wide else None, "dgamma": dgamma}


def _sort(c, ids):
    n, align, cap = c["experts"], c["align"], _capacity(c)
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < n), flat, n)
    counts = torch.zeros(n + 1, dtype=torch.int64, device=key.device).scatter_add_(0, key, torch.ones_like(key))
    padded = (counts + align - 1) // align * align
    offsets = torch.cumsum(padded, 0) - padded          # one start per expert, then the rows' number
    order = torch.argsort(key, stable=True)
    sorted_key = key[order]
    rank = torch.arange(key.numel(), device=key.device) - (torch.cumsum(counts, 0) - counts)[sorted_key]
    pos = torch.empty_like(key)
    pos[order] = torch.where(sorted_key < n, offsets[sorted_key] + rank, -1)
    src = torch.full((cap + 1,), -1, dtype=torch.int64, device=key.device)
    src[torch.where(pos >= 0, pos, cap)] = torch.arange(key.numel(), device=key.device)
    return offsets.int(), pos.view(ids.shape).int(), src[:cap].int()


def _rows_of(y, pos):
    """y's row for every assignment, in FP32, zero where it was dropped."""
    r = y[pos.clamp_min(0).long()].float()
    return torch.where((pos >= 0)[..., None], r, 0)


def _scatter(values, src):
    """values [tokens * k, cols] or [tokens, cols] rows in sorted order, zero in padding rows."""
    return torch.where((src >= 0)[:, None], values, torch.zeros((), dtype=values.dtype, device=values.device))


def _moe_fwd(s):
    c = s["case"]
    offsets, pos, src = _sort(c, s["ids"])
    x = s["x"]
    if c["f8"] == "mx":
        x = (x.view(torch.float8_e4m3fn).float() * _pow2(s["scales"]).repeat_interleave(32, 1)).to(torch.bfloat16)
    elif c["f8"] == "row":
        x = (x.view(torch.float8_e4m3fn).float() * s["scales"][:, None]).to(torch.bfloat16)
    rows = _scatter(x[src.clamp_min(0).long() // c["k"]], src)
    out = (_rows_of(s["y"], pos) * s["weights"][..., None]).sum(1).to(torch.bfloat16)
    return {"offsets": offsets, "pos": pos, "src": src, "rows": rows, "out": out}


def _moe_bwd(s):
    k = s["case"]["k"]
    a = s["src"].clamp_min(0).long()
    dout = s["dout"].float()
    dy = _scatter((dout[a // k] * s["weights"].reshape(-1)[a][:, None]).to(torch.bfloat16), s["src"])
    dw = (_rows_of(s["y"], s["pos"]) * dout[:, None, :]).sum(2)
    dx = _rows_of(s["dx_rows"], s["pos"]).sum(1).to(torch.bfloat16)
    return {"dy": dy, "dw": dw, "dx": dx}


def _philox(c0, c1, c2, c3, seed):
    """Philox4x32-10 of counters (int64 tensors below 2^32) under the key `seed`."""
    mask = 0xFFFFFFFF
    k0, k1 = seed & mask, seed >> 32 & mask
    lo = lambda a, m: ((a & 0xFFFF) * m + (((a >> 16) * m & 0xFFFF) << 16)) & mask  # noqa: E731
    hi = lambda a, m: ((a >> 16) * m + ((a & 0xFFFF) * m >> 16)) >> 16  # noqa: E731
    for _ in range(10):
        h0, l0, h1, l1 = hi(c0, 0xD2511F53), lo(c0, 0xD2511F53), hi(c2, 0xCD9E8D57), lo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    return torch.stack((c0, c1, c2, c3), 1).reshape(-1)


def _stochastic(a, r16, mantissa, lowest, steps):
    """The code of a >= 0 in an 8-bit float with `mantissa` bits, smallest
    normal 2^lowest and subnormal step 1/steps: up where r16 < the 16-bit
    fraction of a's distance to the next value."""
    u = a.view(torch.int32)
    drop = 23 - mantissa
    t = (u >> (drop - 16)) & 0xFFFF
    code = (u >> drop) - ((127 + lowest - 1) << mantissa)
    q = a * steps
    f = torch.floor(q)
    small = a < 2.0 ** lowest
    t = torch.where(small, ((q - f) * 65536).int(), t)
    code = torch.where(small, f.int(), code)
    return code + (r16 < t).int()


def _adamw(s):
    c = s["case"]
    w, m, v = s["w"], s["m"], s["v"]
    if c["states"] == "f8":
        m = (m.view(torch.float8_e4m3fn).float().view(-1, STATE_BLOCK) * s["ms"][:, None]).view(-1)
        v = (v.view(torch.float8_e5m2).float().view(-1, STATE_BLOCK) * s["vs"][:, None]).view(-1)
    g = s["g"].float() * s["scale"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * (1 - BETA2) * g
    new = w * (1 - LR * DECAY) - (m / (torch.sqrt(v) * (1 / math.sqrt(1 - BETA2 ** STEP)) + ADAM_EPS)) * (LR / (1 - BETA1 ** STEP))
    w.copy_(new)
    s["w16"].copy_(new)
    if c["states"] == "f32":
        s["m"].copy_(m)
        s["v"].copy_(v)
        return _adamw_out(s)
    quads = w.numel() // 4
    per = torch.tensor([(n + STATE_BLOCK - 1) // STATE_BLOCK * (STATE_BLOCK // 4) for n in s["sizes"]], device=DEV)
    which = torch.repeat_interleave(torch.arange(len(s["sizes"]), device=DEV), per, output_size=quads)
    at = torch.arange(quads, device=DEV) - (torch.cumsum(per, 0) - per)[which]
    r = _philox(at & 0xFFFFFFFF, at >> 32, which, torch.full_like(at, STEP), s["seed"])
    for x, code, scale, top, draws, kind in ((m, "m", "ms", 448, r & 0xFFFF, (3, -6, 512.0)), (v, "v", "vs", 57344, r >> 16, (2, -14, 65536.0))):
        b = x.view(-1, STATE_BLOCK)
        s[scale].copy_((b.abs().amax(1) / top).clamp_min(TINY))
        a = (b.abs() * (1 / s[scale])[:, None]).clamp_max(top).view(-1)
        q = _stochastic(a, draws.int(), *kind)
        q = q | ((x < 0).int() << 7) if code == "m" else torch.where(x > 0, q.clamp_min(1), q)
        s[code].copy_(q)
    return _adamw_out(s)


def _adamw_out(s):
    o = {"w": s["w"], "w16": s["w16"], "m": s["m"], "v": s["v"]}
    if s["case"]["states"] == "f8":
        o["m"], o["v"] = s["m"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e5m2)
        o["ms"], o["vs"] = s["ms"], s["vs"]
    return o


PLAIN = {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "moe_fwd": _moe_fwd, "moe_bwd": _moe_bwd, "adamw": _adamw}


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """The outputs in float64.  What is rounded to 8 bits has no such value
    (None); a sum that the operator stores in BF16 and works on from there is
    rounded there."""
    s = prepare(case, seed)
    op = case["op"]
    d = lambda t: t.double()  # noqa: E731
    if op == "norm_fwd":
        h = d(s["x"])
        if s["res"] is not None:
            h = d((h + d(s["res"])).to(s["res"].dtype))
        ms = (h ** 2).sum(1) / case["cols"]
        r = (ms + EPS) ** -0.5
        n = h * torch.outer(r, d(s["gain"]))
        o = {"h": None if s["res"] is None else h, "rstd": r, "y": n if case["y"] and case["f8"] == "none" else None}
        if case["f8"] == "mx":
            top = n.reshape(case["rows"], -1, 32).abs().amax(2)
            o["scales"] = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(-127, 127))
        elif case["f8"] == "row":
            o["scales"] = n.abs().amax(1) / 448
        if case["f8"] != "none":
            o["codes"] = None
        return o
    if op == "norm_bwd":
        h, dy, r = d(s["h"]), d(s["dy"]), d(s["rstd"])
        gain = d(s["gain"])
        dot = torch.mv(dy * h, gain)                                # sum of dy * gain * h over a row
        dh = dy * torch.outer(r, gain) - h * (r ** 3 * dot / case["cols"])[:, None]
        if s["dres"] is not None:
            dh = dh + d(s["dres"])
        return {"dh": dh, "dx": dh if s["h"].dtype == torch.float32 else None, "dgamma": torch.mv((dy * h).T, r)}
    if op == "moe_fwd":
        k, h, ids = case["k"], case["cols"], s["ids"].reshape(-1).tolist()
        # place by place, as the definition has it
        starts, rows = [0], [[] for _ in range(case["experts"])]
        for a, e in enumerate(ids):
            if 0 <= e < case["experts"]:
                rows[e].append(a)
        pos, src = [-1] * len(ids), [-1] * _capacity(case)
        for e, members in enumerate(rows):
            for i, a in enumerate(members):
                pos[a], src[starts[e] + i] = starts[e] + i, a
            starts.append(starts[e] + -(-len(members) // case["align"]) * case["align"])
        x = s["x"]
        if case["f8"] == "mx":
            x = d(x.view(torch.float8_e4m3fn)).reshape(-1, h // 32, 32) * torch.exp2(d(s["scales"]) - 127)[:, :, None]
        elif case["f8"] == "row":
            x = d(x.view(torch.float8_e4m3fn)) * d(s["scales"])[:, None]
        x = torch.cat((d(x).reshape(-1, h), torch.zeros((1, h), dtype=torch.float64, device=DEV)))
        src = torch.tensor(src, device=DEV)
        out = torch.zeros((case["tokens"], h), dtype=torch.float64, device=DEV)
        live = src >= 0
        out.index_add_(0, src[live] // k, d(s["y"])[live] * d(s["weights"]).reshape(-1)[src[live]][:, None])
        i32 = lambda v: torch.as_tensor(v, device=DEV).int()  # noqa: E731
        return {"offsets": i32(starts), "pos": i32(pos).view(-1, k), "src": src.int(),
                "rows": x[torch.where(live, src // k, case["tokens"])], "out": out}
    if op == "moe_bwd":
        k, t, h = case["k"], case["tokens"], case["cols"]
        live = s["src"] >= 0
        a = s["src"][live].long()
        dout, w = d(s["dout"]), d(s["weights"]).reshape(-1)
        dy = torch.zeros((s["src"].numel(), h), dtype=torch.float64, device=DEV)
        dy[live] = dout[a // k] * w[a][:, None]
        dw = torch.zeros(t * k, dtype=torch.float64, device=DEV)
        dw[a] = (d(s["y"])[live] * dout[a // k]).sum(1)
        dx = torch.zeros((t, h), dtype=torch.float64, device=DEV).index_add_(0, a // k, d(s["dx_rows"])[live])
        return {"dy": dy, "dw": dw.view(t, k), "dx": dx}
    m, v = s["m"], s["v"]
    if case["states"] == "f8":
        m = d(m.view(torch.float8_e4m3fn)) * d(s["ms"]).repeat_interleave(STATE_BLOCK)
        v = d(v.view(torch.float8_e5m2)) * d(s["vs"]).repeat_interleave(STATE_BLOCK)
    g = d(s["g"]) * GRAD_SCALE
    m = BETA1 * d(m) + (1 - BETA1) * g
    v = BETA2 * d(v) + (1 - BETA2) * g ** 2
    w = d(s["w"])
    w = w - LR * DECAY * w - LR * (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)) ** 0.5 + ADAM_EPS)
    if case["states"] == "f32":
        return {"w": w, "w16": w, "m": m, "v": v}
    top = lambda x: x.abs().reshape(-1, STATE_BLOCK).amax(1)  # noqa: E731
    return {"w": w, "w16": w, "m": None, "v": None, "ms": top(m) / 448, "vs": top(v) / 57344}
