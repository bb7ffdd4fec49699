"""Cases for the operators around the MoE layer's GEMMs: their inputs, their plain forms and their exact values.

Four families, each reached through the package's public functions:

* ``norm`` / ``norm_bwd``: the layer norm (or root mean square norm) at the layer's entry and its backward pass, from the
  saved input or from the 8-bit checkpoint of the normalised rows;
* ``ckpt`` / ``ckpt_swiglu`` / ``ckpt_combine``: activation checkpoints in 8 bits (E4M3 codes, one power-of-two scale per
  1x128 tile) and the two backward kernels that read them;
* ``w4``: the experts' products with 4-bit weights (E2M1 codes, one power-of-two scale per 32 inputs) for decode batches.

Sizes are those of the DeepSeek-V3-shaped layer that the package's configurations hold (hidden 7168, 256 routed + 1 shared
experts of width 2048, top-8), of its tiny configuration, and odd ones between.
"""
import math

import torch

own = False

DEV = "cuda"
TILE = 128   # columns per scale of an 8-bit checkpoint
GROUP = 32   # inputs per scale of a 4-bit weight
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


def listed():
    return [
        # the norm of one decoded token: latency only
        {"name": "norm_decode_T1", "op": "norm", "T": 1, "d": 7168, "dtype": "bf16", "rms": True, "bias": False, "ckpt": False,
         "pad": 0},
        # a training batch: the norm also writes its 8-bit checkpoint, which is read back as a backward pass does
        {"name": "norm_train_T4096", "op": "norm", "T": 4096, "d": 7168, "dtype": "bf16", "rms": True, "bias": False,
         "ckpt": True, "pad": 0},
        # ragged rows of a width that fills no vector, inside a wider matrix
        {"name": "norm_odd_f32", "op": "norm", "T": 2500, "d": 1023, "dtype": "f32", "rms": False, "bias": True, "ckpt": False,
         "pad": 5},
        # the layer norm's backward pass over a training batch, with the weight's and the bias's gradient
        {"name": "norm_bwd_T4096", "op": "norm_bwd", "T": 4096, "d": 7168, "dtype": "bf16", "rms": False, "bias": True,
         "ckpt": False, "grad": "f32"},
        # the same for the largest training batch, from the 8-bit checkpoint
        {"name": "norm_bwd_ckpt_T16384", "op": "norm_bwd", "T": 16384, "d": 7168, "dtype": "bf16", "rms": True, "bias": False,
         "ckpt": True, "grad": "bf16"},
        # the routed and shared experts' gate | up products of a training batch, packed and read back
        {"name": "ckpt_pack_T4096", "op": "ckpt", "rows": 36864, "cols": 4096, "dtype": "f32"},
        # the SwiGLU backward of the tiny configuration (64 tokens, 2 + 1 experts each, width 64)
        {"name": "ckpt_swiglu_tiny", "op": "ckpt_swiglu", "rows": 192, "inter": 64},
        # the SwiGLU backward of a training batch (4096 tokens, 8 + 1 experts each)
        {"name": "ckpt_swiglu_T4096", "op": "ckpt_swiglu", "rows": 36864, "inter": 2048},
        # the combine's and the router's gradients of that batch, from the expert outputs in 8 bits
        {"name": "ckpt_combine_T4096", "op": "ckpt_combine", "T": 4096, "d": 7168, "experts": 256, "top_k": 8},
        # one decoded token through the gate/up projections of its 8 experts and the shared one
        {"name": "w4_gate_up_T1", "op": "w4", "T": 1, "d": 7168, "inter": 2048, "experts": 256, "top_k": 8, "zipf": 0.0,
         "down": False},
        # 16 tokens through the down projections
        {"name": "w4_down_T16", "op": "w4", "T": 16, "d": 7168, "inter": 2048, "experts": 256, "top_k": 8, "zipf": 0.0,
         "down": True},
        # a full decode batch with skewed routing: nearly every expert is read, a few hold many rows
        {"name": "w4_gate_up_T256", "op": "w4", "T": 256, "d": 7168, "inter": 2048, "experts": 256, "top_k": 8, "zipf": 1.1,
         "down": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "ckpt", "ckpt_swiglu", "ckpt_combine", "w4", "w4"])
    if op in ("norm", "norm_bwd"):
        d = _log_int(rng, 16, 16384)
        T = _log_int(rng, 1, min(16384, 16384 * 7168 // d))
        rms = rng.random() < 0.5
        c = {"op": op, "T": T, "d": d, "dtype": rng.choice(["bf16", "f32"]), "rms": rms,
             "bias": not rms and rng.random() < 0.7, "ckpt": rng.random() < 0.5}
        if op == "norm":
            c["pad"] = rng.choice([0, 0, 8, rng.randint(1, 200)])
        else:
            c["grad"] = rng.choice(["bf16", "f32"])
        return c
    if op == "ckpt":
        cols = _log_int(rng, 16, 8192)
        return {"op": op, "rows": _log_int(rng, 1, 36864 * 4096 // cols // 4), "cols": cols, "dtype": rng.choice(["bf16", "f32"])}
    if op == "ckpt_swiglu":
        inter = 4 * _log_int(rng, 4, 512)
        return {"op": op, "rows": _log_int(rng, 1, 36864), "inter": inter}
    if op == "ckpt_combine":
        E = 4 * rng.randint(4, 64)
        return {"op": op, "T": _log_int(rng, 1, 4096), "d": 8 * _log_int(rng, 8, 896), "experts": E, "top_k": rng.randint(1, 8)}
    E = 4 * rng.randint(4, 64)
    return {"op": "w4", "T": _log_int(rng, 1, 256), "d": 32 * _log_int(rng, 4, 224), "inter": 32 * _log_int(rng, 2, 64),
            "experts": E, "top_k": rng.randint(1, 8), "zipf": rng.choice([0.0, 0.6, 1.1]), "down": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _residual(g, T, d, dtype):
    """Rows as a residual stream has them: about unit normal, a row mean off zero, a few channels much larger."""
    big = 1.0 + 20.0 * (torch.rand(d, generator=g, device=DEV) < 0.002).float()
    return ((_randn(g, T, d) + 0.3) * big).to(dtype)


def _tile_exponents(x):
    """The smallest k with max |x| <= 448 * 2^k of each 1x128 tile, within [-127, 127]; 0 for a tile of zeros."""
    cols = x.shape[1]
    t = torch.nn.functional.pad(x, (0, -cols % TILE)).view(x.shape[0], -1, TILE).abs().amax(-1)
    m, e = torch.frexp(t)
    k = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-127, 127)
    return torch.where(t == 0, torch.zeros_like(k), k)


def _pack(x):
    """Codes [rows, cols] and scale codes [rows, ceil(cols / 128)] of an 8-bit checkpoint."""
    k = _tile_exponents(x)
    s = torch.exp2(-k.float()).repeat_interleave(TILE, 1)[:, :x.shape[1]]
    return (x * s).to(torch.float8_e4m3fn).view(torch.uint8), (k + 127).to(torch.uint8)


def _values(q, s):
    """What the codes of an 8-bit checkpoint stand for, in float32."""
    p = torch.exp2(s.float() - 127.0).repeat_interleave(TILE, 1)[:, :q.shape[1]]
    return q.view(torch.float8_e4m3fn).float() * p


def _routing(g, T, E, K, zipf):
    """K distinct experts of each token by popularity rank^-zipf, sorted by expert: offsets of the routed experts and the
    shared one, the token of each sorted row, and the row of each (token, k)."""
    rank = torch.randperm(E, generator=g, device=DEV).float() + 1.0
    gumbel = -torch.log(-torch.log(torch.rand((T, E), generator=g, device=DEV).clamp(1e-20, 1.0 - 1e-7)))
    idx = (gumbel - zipf * torch.log(rank)).topk(K, 1).indices
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    offs = torch.zeros(E + 2, dtype=torch.int64, device=DEV)
    offs[1:E + 1] = counts.cumsum(0)
    offs[E + 1] = T * K + T
    token = torch.cat([order // K, torch.arange(T, device=DEV)])
    pos = torch.empty(T * K, dtype=torch.int64, device=DEV)
    pos[order] = torch.arange(T * K, device=DEV)
    return idx.to(torch.int32), offs.to(torch.int32), token.to(torch.int32), pos.view(T, K).to(torch.int32)


def _w4_weights(g, G, n, k, std):
    """Weights in 4 bits as a quantiser leaves them: nibbles spread like a normal's, scale codes about the weights' size."""
    q = torch.arange(256, device=DEV, dtype=torch.float32).add(0.5).div(256)
    z = math.sqrt(2.0) * torch.erfinv(2.0 * q - 1.0) * 2.0  # quantiles of a normal in units of the group's scale
    mag = torch.bucketize(z.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV))
    nib = (mag + 8 * (z < 0)).to(torch.uint8)
    q4 = torch.empty((G, n, k // 2), dtype=torch.uint8, device=DEV)
    for a in range(0, G, 32):
        b = min(G, a + 32)
        lo = torch.randint(0, 256, (b - a, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
        hi = torch.randint(0, 256, (b - a, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
        q4[a:b] = nib[lo.int()] | (nib[hi.int()] << 4)
    e = 127 + int(round(math.log2(std / 2.0)))
    s = torch.randint(e - 1, e + 2, (G, n, k // GROUP), generator=g, device=DEV, dtype=torch.uint8)
    return q4, s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        T, d, dt = case["T"], case["d"], DTYPES[case["dtype"]]
        s["w"] = 1.0 + 0.2 * _randn(g, d)
        s["b"] = 0.1 * _randn(g, d) if case["bias"] else None
        if op == "norm":
            s["x"] = _residual(g, T, d + case["pad"], dt)[:, :d]
            return s
        s["dy"] = (0.02 * _randn(g, T, d)).to(DTYPES[case["grad"]])
        x = _residual(g, T, d, dt)
        xf = x.float()
        mean = torch.zeros(T, device=DEV) if case["rms"] else xf.mean(1)
        rstd = torch.rsqrt((xf - mean[:, None]).square().mean(1) + EPS)
        s["mean"], s["rstd"] = (None if case["rms"] or case["ckpt"] else mean), rstd
        if case["ckpt"]:
            s["x"] = None
            s["q"], s["s"] = _pack((xf - mean[:, None]) * rstd[:, None])
        else:
            s["x"] = x
    elif op == "ckpt":
        r, c = case["rows"], case["cols"]
        x = _randn(g, r, c) * torch.exp(0.5 * _randn(g, r, 1))
        s["x"] = x.to(DTYPES[case["dtype"]])
    elif op == "ckpt_swiglu":
        r, i = case["rows"], case["inter"]
        s["q"], s["s"] = _pack(_randn(g, r, 2 * i) * 0.6)
        s["dh"] = _randn(g, r, i) * 0.05
    elif op == "ckpt_combine":
        T, d, E, K = case["T"], case["d"], case["experts"], case["top_k"]
        s["idx"], _, _, s["pos"] = _routing(g, T, E, K, 0.0)
        s["scores"] = torch.sigmoid(0.5 * _randn(g, T, E))
        v = s["scores"].gather(1, s["idx"].long())
        s["gate"] = v / v.sum(1, keepdim=True)
        s["q"], s["s"] = _pack((_randn(g, T * K, d) * 0.1))
        s["d_out"] = _randn(g, T, d).bfloat16()
    else:
        T, d, inter, E, K = case["T"], case["d"], case["inter"], case["experts"], case["top_k"]
        _, offs, token, _ = _routing(g, T, E, K, case["zipf"])
        s["offs"] = offs
        rows = T * (K + 1)
        lens = (offs[1:] - offs[:-1]).long()
        # the plain form's plan: the groups that hold rows, each row's place among them
        active = lens.nonzero().view(-1)
        s["active"], s["most"] = active, int(lens.max())
        group = torch.repeat_interleave(torch.arange(len(active), device=DEV), lens[active])
        s["slot"] = group * s["most"] + torch.arange(rows, device=DEV) - offs[:-1].long()[active][group]
        if case["down"]:
            s["token"] = None
            s["x"] = (_randn(g, rows, inter) * 0.1).bfloat16()
            s["q"], s["s"] = _w4_weights(g, E + 1, d, inter, 0.006)
        else:
            s["token"] = token
            s["x"] = _randn(g, T, d).bfloat16()
            s["q"], s["s"] = _w4_weights(g, E + 1, 2 * inter, d, 0.006)
    return s


# ------------------------------------------------------------------ one pass


def _norm_plain(s):
    c = s["case"]
    x = s["x"].float()
    mean = torch.zeros(x.shape[0], device=x.device) if c["rms"] else x.mean(1)
    xc = x - mean[:, None]
    rstd = torch.rsqrt(xc.square().mean(1) + EPS)
    xhat = xc * rstd[:, None]
    y = xhat * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    out = [y.to(s["x"].dtype), rstd]
    if not c["rms"]:
        out.append(mean)
    if c["ckpt"]:
        out.append(_values(*_pack(xhat)).bfloat16())
    return out


def _norm_bwd_plain(s):
    c = s["case"]
    dy = s["dy"].float()
    if c["ckpt"]:
        xhat = _values(s["q"], s["s"])
    else:
        x = s["x"].float()
        xhat = (x if s["mean"] is None else x - s["mean"][:, None]) * s["rstd"][:, None]
    gy = dy * s["w"]
    dx = gy - xhat * (gy * xhat).mean(1, keepdim=True)
    if not c["rms"]:
        dx = dx - gy.mean(1, keepdim=True)
    dx = (dx * s["rstd"][:, None]).to(s["dy"].dtype)
    dw = (dy * xhat).sum(0)
    return [dx, dw] if s["b"] is None else [dx, dw, dy.sum(0)]


def _swiglu_bwd_plain(s):
    i = s["case"]["inter"]
    v = _values(s["q"], s["s"])
    a, c, dh = v[:, :i], v[:, i:], s["dh"]
    sg = torch.sigmoid(a)
    dac = torch.cat([dh * c * sg * (1.0 + a * (1.0 - sg)), dh * a * sg], 1)
    return [dac.bfloat16(), (a * sg * c).bfloat16()]


def _combine_bwd_plain(s):
    T, K = s["idx"].shape
    idx, pos = s["idx"].long(), s["pos"].long()
    d_out = s["d_out"].float()
    dy = torch.empty((T * (K + 1), d_out.shape[1]), dtype=torch.bfloat16, device=DEV)
    dy[pos.reshape(-1)] = (s["gate"][:, :, None] * d_out[:, None, :]).bfloat16().view(T * K, -1)
    dy[T * K:] = s["d_out"]
    dg = (_values(s["q"], s["s"])[pos.reshape(-1)].view(T, K, -1) * d_out[:, None, :]).sum(2)
    v = s["scores"].gather(1, idx)
    du = v * (1.0 - v) * (dg - (s["gate"] * dg).sum(1, keepdim=True)) / v.sum(1, keepdim=True)
    du_row = torch.empty(T * K, device=DEV)
    du_row[pos.reshape(-1)] = du.reshape(-1)
    return [dy, du, du_row]


def _w4_plain(s):
    c = s["case"]
    T, K = c["T"], c["top_k"]
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    q, sc = s["q"][s["active"]], s["s"][s["active"]]
    A, n, kb = q.shape
    w = torch.empty((A, n, kb, 2), device=DEV)
    w[..., 0] = lut[(q & 15).int()]
    w[..., 1] = lut[(q >> 4).int()]
    w = w.view(A, n, sc.shape[2], GROUP).mul_(torch.exp2(sc.float() - 127.0)[..., None]).view(A, n, 2 * kb)
    x = s["x"] if s["token"] is None else s["x"][s["token"].long()]
    xg = torch.zeros((A * s["most"], 2 * kb), device=DEV)
    xg[s["slot"]] = x.float()
    out = torch.bmm(w, xg.view(A, s["most"], -1).transpose(1, 2).contiguous())
    out = out.transpose(1, 2).reshape(A * s["most"], n)[s["slot"]]
    if c["down"]:
        return [out[:T * K].bfloat16(), out[T * K:]]
    a, u = out[:, :n // 2], out[:, n // 2:]
    return (a * torch.sigmoid(a) * u).bfloat16()


PLAIN = {"norm": _norm_plain, "norm_bwd": _norm_bwd_plain, "ckpt_swiglu": _swiglu_bwd_plain,
         "ckpt_combine": _combine_bwd_plain, "w4": _w4_plain,
         "ckpt": lambda s: _values(*_pack(s["x"].float())).bfloat16()}


def _own(s):
    import sparse_moe_layer_sigmoid_amd as M
    c = s["case"]
    op = c["op"]
    if op == "norm":
        y, mean, rstd, ck = M.moe_norm(s["x"], s["w"], s["b"], eps=EPS, rms=c["rms"], want_stats=True, checkpoint=c["ckpt"])
        out = [y, rstd] if c["rms"] else [y, rstd, mean]
        return out + [M.fp8_ckpt_unpack(*ck)] if c["ckpt"] else out
    if op == "norm_bwd":
        ck = (s["q"], s["s"]) if c["ckpt"] else None
        dx, dw, db = M.moe_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], rms=c["rms"], checkpoint=ck,
                                         want_dbias=c["bias"], out_dtype=s["dy"].dtype)
        return [dx, dw] if db is None else [dx, dw, db]
    if op == "ckpt":
        return M.fp8_ckpt_unpack(*M.fp8_ckpt_pack(s["x"]))
    if op == "ckpt_swiglu":
        return list(M.moe_swiglu_backward_ckpt(s["q"], s["s"], s["dh"]))
    if op == "ckpt_combine":
        return list(M.moe_combine_backward_ckpt(s["d_out"], s["q"], s["s"], s["idx"], s["gate"], s["scores"], s["pos"]))
    T, K, E = c["T"], c["top_k"], c["experts"]
    rows = T * (K + 1)
    if c["down"]:
        y = torch.empty((T * K, c["d"]), dtype=torch.bfloat16, device=DEV)
        ysh = torch.empty((T, c["d"]), dtype=torch.float32, device=DEV)
        M.moe_w4_gemm(s["x"], s["q"], s["s"], s["offs"], 0, E + 1, rows, y, out_tail=ysh, tail_groups=1)
        return [y, ysh]
    h = torch.empty((rows, c["inter"]), dtype=torch.bfloat16, device=DEV)
    return M.moe_w4_gemm(s["x"], s["q"], s["s"], s["offs"], 0, E + 1, rows, h, a_rows=s["token"], swiglu=True)


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without


def _active(E, K, T, zipf):
    """Expected number of routed experts that T tokens reach, by popularity rank^-zipf."""
    p = [r ** -zipf for r in range(1, E + 1)]
    lo, hi = 0.0, 1e9
    for _ in range(100):  # inclusion of expert e by one token is about 1 - exp(-c p_e), the sum being K
        mid = (lo + hi) / 2
        if sum(1.0 - math.exp(-mid * v) for v in p) < K:
            lo = mid
        else:
            hi = mid
    return sum(1.0 - math.exp(-lo * v * T) for v in p)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, d, T = case["T"] * case["d"], case["d"], case["T"]
        es = 2 if case["dtype"] == "bf16" else 4
        ck = n + T * -(-d // TILE)
        vec = 4 * d * (2 if case["bias"] else 1) + 4 * T * (1 if case["rms"] else 2)
        if op == "norm":
            return {"bytes": 2 * n * es + vec + (2 * ck + 2 * n if case["ckpt"] else 0), "flops": 8 * n}
        gs = 2 if case["grad"] == "bf16" else 4
        return {"bytes": 2 * n * gs + (ck if case["ckpt"] else n * es) + 2 * vec, "flops": 14 * n}
    if op == "ckpt":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + 2 * (n + case["rows"] * -(-case["cols"] // TILE)) + 2 * n,
                "flops": 4 * n}
    if op == "ckpt_swiglu":
        n = case["rows"] * case["inter"]
        return {"bytes": 2 * n + case["rows"] * -(-2 * case["inter"] // TILE) + 4 * n + 6 * n, "flops": 20 * n}
    if op == "ckpt_combine":
        T, K, d = case["T"], case["top_k"], case["d"]
        return {"bytes": T * d * 2 + T * K * (d + -(-d // TILE)) + T * (K + 1) * d * 2 + T * K * 20, "flops": 4 * T * K * d}
    T, K, E = case["T"], case["top_k"], case["experts"]
    n, k = (case["d"], case["inter"]) if case["down"] else (2 * case["inter"], case["d"])
    weights = (_active(E, K, T, case["zipf"]) + 1) * n * (k // 2 + k // GROUP)
    rows = T * (K + 1)
    io = rows * k * 2 + T * K * n * 2 + T * n * 4 if case["down"] else T * k * 2 + rows * n
    return {"bytes": weights + io, "flops": 2.0 * rows * n * k}


# ------------------------------------------------------------------ the definitions in 64 bits


def _e4m3_64(v):
    """v rounded to the E4M3 grid, half to even: eight steps to a binade, 2^-9 below 2^-6."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=v.device), e.clamp_min(-6) - 3)
    return torch.round(v / step) * step


def _ckpt_64(x):
    """x through the 8-bit checkpoint's definition, in 64 bits."""
    r, c = x.shape
    n = -(-c // TILE)
    p = torch.zeros((r, n * TILE), dtype=torch.float64, device=x.device)
    p[:, :c] = x
    p = p.view(r, n, TILE)
    amax = p.abs().amax(2, keepdim=True)
    k = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.full_like(amax, 448.0)) / 448.0)).clamp(-127, 127)
    s = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=x.device), k)
    return (_e4m3_64(p / s) * s).view(r, n * TILE)[:, :c]


def _decode_64(q, s):
    """E4M3 codes and scale codes -> values, field by field."""
    c = q.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.pow(2.0, (e - 7).double()))
    v = torch.where(c >= 128, -v, v)
    cols = torch.arange(q.shape[1], device=q.device) // TILE
    return v * torch.pow(2.0, s.double()[:, cols] - 127.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = lambda t: t.to(torch.float64)  # noqa: E731
    if op == "norm":
        outs = []
        step = max(1, (1 << 26) // case["d"])
        for a in range(0, case["T"], step):
            x = f64(s["x"][a:a + step])
            mean = x.mean(1, keepdim=True) * (0.0 if case["rms"] else 1.0)
            rstd = ((x - mean) ** 2).mean(1, keepdim=True).add(EPS) ** -0.5
            xhat = (x - mean) * rstd
            y = xhat * f64(s["w"]) + (0.0 if s["b"] is None else f64(s["b"]))
            o = [y, rstd[:, 0]] + ([] if case["rms"] else [mean[:, 0]])
            outs.append(o + ([_ckpt_64(xhat)] if case["ckpt"] else []))
        return [torch.cat(t) for t in zip(*outs)]
    if op == "norm_bwd":
        dxs, dw, db = [], 0.0, 0.0
        step = max(1, (1 << 26) // case["d"])
        for a in range(0, case["T"], step):
            r = slice(a, a + step)
            dy, rstd = f64(s["dy"][r]), f64(s["rstd"][r])[:, None]
            if case["ckpt"]:
                xhat = _decode_64(s["q"][r], s["s"][r])
            else:
                xhat = (f64(s["x"][r]) - (0.0 if s["mean"] is None else f64(s["mean"][r])[:, None])) * rstd
            gy = dy * f64(s["w"])
            along = (gy * xhat).mean(1, keepdim=True) * xhat
            dxs.append(rstd * (gy - along - (0.0 if case["rms"] else gy.mean(1, keepdim=True))))
            dw, db = dw + (dy * xhat).sum(0), db + dy.sum(0)
        return [torch.cat(dxs), dw] + ([] if s["b"] is None else [db])
    if op == "ckpt":
        step = max(1, (1 << 26) // case["cols"])
        return torch.cat([_ckpt_64(f64(s["x"][a:a + step])).float() for a in range(0, case["rows"], step)]).double()
    if op == "ckpt_swiglu":
        i, dac, h = case["inter"], [], []
        step = max(1, (1 << 25) // i)
        for a0 in range(0, case["rows"], step):
            r = slice(a0, a0 + step)
            v, dh = _decode_64(s["q"][r], s["s"][r]), f64(s["dh"][r])
            a, c = v[:, :i], v[:, i:]
            sg = 1.0 / (1.0 + torch.exp(-a))
            dac.append(torch.cat([dh * c * (sg + a * sg * (1.0 - sg)), dh * (a * sg)], 1))
            h.append(a * sg * c)
        return [torch.cat(dac), torch.cat(h)]
    if op == "ckpt_combine":
        T, K = s["idx"].shape
        dy = torch.zeros((T * (K + 1), case["d"]), dtype=torch.float64, device=DEV)
        dg = torch.zeros((T, K), dtype=torch.float64, device=DEV)
        d_out, gate, p = f64(s["d_out"]), f64(s["gate"]), s["pos"].long()
        for k in range(K):
            dy[p[:, k]] = gate[:, k:k + 1] * d_out
            dg[:, k] = (_decode_64(s["q"][p[:, k]], s["s"][p[:, k]]) * d_out).sum(1)
        dy[T * K:] = d_out
        v = f64(s["scores"]).gather(1, s["idx"].long())
        S = v.sum(1, keepdim=True)
        du = v * (1.0 - v) / S * (dg - (gate * dg).sum(1, keepdim=True))
        row = torch.zeros(T * K, dtype=torch.float64, device=DEV)
        row[p.reshape(-1)] = du.reshape(-1)
        return [dy, du, row]
    T, K = case["T"], case["top_k"]
    offs = s["offs"].tolist()
    mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    parts = []
    for g in range(case["experts"] + 1):
        a, b = offs[g], offs[g + 1]
        if a == b:
            continue
        x = f64(s["x"][a:b] if s["token"] is None else s["x"][s["token"][a:b].long()])
        c = s["q"][g].int()
        nib = torch.stack([c & 15, c >> 4], -1).view(c.shape[0], -1)
        w = mag[nib & 7] * torch.where(nib >= 8, -1.0, 1.0)
        w = w * torch.pow(2.0, f64(s["s"][g]) - 127.0).repeat_interleave(GROUP, 1)
        parts.append(x @ w.t().contiguous())
    out = torch.cat(parts)
    if case["down"]:
        return [out[:T * K], out[T * K:]]
    n = out.shape[1] // 2
    return out[:, :n] / (1.0 + torch.exp(-out[:, :n])) * out[:, n:]
