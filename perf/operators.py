"""Measured cases of the 16-bit and 8-bit-integer expert products and of the expert weights' AdamW step.

Three operators, each on the shapes that an expert layer meets:

* grouped bf16 products of a dropless mixture-of-experts layer: Y_g = X_g W_g^T (forward),
  dX_g = dY_g W_g (dgrad) and dW_g = dY_g^T X_g (wgrad) over the expert's real rows;
* grouped products of 8-bit integers with one scale per token and one per output channel, with the
  quantiser that makes the tokens' codes (from a tensor, or from the SwiGLU of a gate|up tensor);
* the AdamW step over a list of tensors with fp32 weights and bf16 copies of them, the moments held in
  fp32 or in 8 bits with a scale per 128 elements.

`run` computes them in plain torch operations, or with `own` set by the library's entry points.
"""
import math

import torch

own = False

TOP = 1.875            # largest value of the second moment's 8-bit code (before its block's scale)
TINY = 2.0 ** -126     # smallest scale of a block


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the smallest layer of the tests: one training pass, bound by launches
        {"name": "bf16 step tiny", "op": "gemm", "dirs": "fdw", "G": 4, "T": 512, "top": 2, "N": 512, "K": 256,
         "skew": 1.0, "out": "bf16"},
        # serving the 64-expert layer: 8 tokens in flight, six experts each, every weight read once
        {"name": "bf16 fwd decode", "op": "gemm", "dirs": "f", "G": 64, "T": 8, "top": 6, "N": 2816, "K": 2048,
         "skew": 0.0, "out": "bf16"},
        # odd sizes: rows, columns and contractions that end inside a tile
        {"name": "bf16 step odd", "op": "gemm", "dirs": "fdw", "G": 7, "T": 5003, "top": 1, "N": 1000, "K": 1112,
         "skew": 1.0, "out": "f32"},
        # training the 64-expert layer's down projection (8192 tokens, top 6)
        {"name": "bf16 step 64 experts", "op": "gemm", "dirs": "fdw", "G": 64, "T": 8192, "top": 6, "N": 2048,
         "K": 1408, "skew": 0.3, "out": "bf16"},
        # training the 16-expert layer's gate and up projection (32768 tokens, top 1): the largest
        {"name": "bf16 step 16 experts", "op": "gemm", "dirs": "fdw", "G": 16, "T": 32768, "top": 1, "N": 16384,
         "K": 5120, "skew": 0.3, "out": "bf16"},
        # serving one GPU's 8 experts, one token each: gate and up projection
        {"name": "int8 decode", "op": "int8", "gated": False, "G": 8, "T": 8, "top": 1, "N": 4096, "K": 7168,
         "skew": 0.0, "out": "bf16"},
        # prefill of the 64-expert layer's gate and up projection
        {"name": "int8 prefill", "op": "int8", "gated": False, "G": 64, "T": 8192, "top": 6, "N": 2816, "K": 2048,
         "skew": 0.3, "out": "bf16"},
        # down projection after SwiGLU with a few tokens in flight
        {"name": "int8 gated down decode", "op": "int8", "gated": True, "G": 64, "T": 21, "top": 6, "N": 2048,
         "K": 1408, "skew": 0.3, "out": "f32"},
        # down projection after SwiGLU, one GPU's 8 experts on 65536 routed rows
        {"name": "int8 gated down prefill", "op": "int8", "gated": True, "G": 8, "T": 65536, "top": 1, "N": 7168,
         "K": 2048, "skew": 0.3, "out": "bf16"},
        # norms, biases and routers: many small tensors of odd lengths
        {"name": "adamw small tensors", "op": "adamw", "bits": 32, "count": 16, "least": 1, "most": 300000,
         "grad": "f32"},
        # the 64-expert layer's two weights with fp32 moments
        {"name": "adamw fp32 moments", "op": "adamw", "bits": 32, "count": 2, "least": 184549376, "most": 369098752,
         "grad": "f32"},
        # one GPU's 8 experts of gate and up weights with 8-bit moments
        {"name": "adamw 8-bit moments", "op": "adamw", "bits": 8, "count": 2, "least": 117440512, "most": 234881024,
         "grad": "bf16"},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    kind = rng.choice(["gemm", "gemm", "int8", "int8", "adamw"])
    if kind == "adamw":
        count = rng.randrange(1, 17)
        most = _log_int(rng, 1000, 300_000_000 // count)
        return {"op": "adamw", "bits": rng.choice([8, 32]), "count": count, "least": _log_int(rng, 1, most),
                "most": most, "grad": rng.choice(["f32", "bf16"])}
    G = _log_int(rng, 1, 96)
    top = rng.randrange(1, min(G, 8) + 1)
    N = _log_int(rng, 128, 8192, 8)
    K = _log_int(rng, 128, 7168, 16)
    while G * N * K > 1.3e9:
        G = max(1, G // 2)
        top = min(top, G)
    most = max(2, int(min(65536 // top, 1.0e12 / (N * K * top))))
    case = {"G": G, "T": _log_int(rng, 1, most), "top": top, "N": N, "K": K,
            "skew": round(rng.uniform(0.0, 1.0), 2), "out": rng.choice(["f32", "bf16"])}
    if kind == "gemm":
        return {"op": "gemm", "dirs": rng.choice(["f", "d", "w", "fdw"]), **case}
    return {"op": "int8", "gated": rng.random() < 0.5, **case}


# -------------------------------------------------------------------------------------------- inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1009 + salt)
    return g


def _randn(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _bf16(shape, gen, std=1.0, slab=64):
    """Normal values in bf16, made a slab of leading rows at a time."""
    out = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    for i in range(0, shape[0], slab):
        n = min(slab, shape[0] - i)
        out[i:i + n] = torch.randn((n, *shape[1:]), generator=gen, device="cuda", dtype=torch.bfloat16) * std
    return out


def _route(case, gen):
    """Group offsets of T tokens' `top` largest router logits, some experts liked more than others."""
    logits = _randn((case["T"], case["G"]), gen) + case["skew"] * _randn((1, case["G"]), gen)
    chosen = logits.topk(case["top"], dim=1).indices
    sizes = torch.bincount(chosen.reshape(-1), minlength=case["G"])
    offs = torch.zeros(case["G"] + 1, device="cuda", dtype=torch.int32)
    offs[1:] = sizes.cumsum(0).to(torch.int32)
    return offs, int(sizes.max())


def _sizes(case):
    """Element counts between least and most, evenly in the logarithm, odd where that leaves room."""
    lo, hi, n = case["least"], case["most"], case["count"]
    if n == 1:
        return [hi]
    return [min(hi, max(lo, round(lo * (hi / lo) ** (i / (n - 1))))) for i in range(n)]


def prepare(case, seed):
    case = dict(case)
    gen = _gen(seed, 1)
    state = {"case": case}
    if case["op"] == "adamw":
        big = case["most"] > 1 << 20
        state.update(step=7, lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1,
                     scale=torch.full((1,), 0.75, device="cuda"))
        lists = {k: [] for k in ("p", "w", "g", "m", "v", "ms", "vs")}
        for n in _sizes(case):
            # weights and gradients of an expert layer: rows of different size, some of them never routed to
            rows = torch.exp(_randn((n // 2048 + 1,), gen)).repeat_interleave(2048)[:n]
            p = _randn((n,), gen, 0.02)
            g = _randn((n,), gen, 1e-3) * rows
            m = _randn((n,), gen, 5e-4) * rows
            v = (_randn((n,), gen, 1e-3) * rows).square_()
            if big:
                g[: n // 64] = 0
                m[: n // 64] = 0
                v[: n // 64] = 0
            lists["p"].append(p)
            lists["w"].append(p.to(torch.bfloat16))
            lists["g"].append(g.to(torch.bfloat16) if case["grad"] == "bf16" else g)
            if case["bits"] == 8:
                mq, ms = _pack_m(m)
                vq, vs = _pack_v(v)
                m, v = mq, vq
                lists["ms"].append(ms)
                lists["vs"].append(vs)
            lists["m"].append(m)
            lists["v"].append(v)
            del rows
        state.update(lists)
        state["table"] = None
        return state
    G, N, K = case["G"], case["N"], case["K"]
    offs, most = _route(case, gen)
    M = case["T"] * case["top"]
    state.update(offs=offs, most=most, M=M)
    if case["op"] == "gemm":
        state["w"] = _bf16((G * N, K), gen, 0.02, 65536)
        state["x"] = _bf16((M, K), gen, 1.0, 65536) if "f" in case["dirs"] or "w" in case["dirs"] else None
        state["dy"] = _bf16((M, N), gen, 1.0, 65536) if "d" in case["dirs"] or "w" in case["dirs"] else None
    else:
        state["qw"] = torch.randint(-127, 128, (G * N, K), generator=gen, device="cuda", dtype=torch.int8)
        state["sw"] = torch.exp(0.3 * _randn((G * N,), gen)) * (0.02 / 73)
        # one token in eight carries a few large channels
        x = _bf16((M, 2 * K if case["gated"] else K), gen, 1.0, 65536)
        x[::8, 5::251] *= 20
        state["x"] = x
    return state


# --------------------------------------------------------------------------------------- plain forms
def _expert_rows(s):
    """[G, most] rows of every expert (clamped), and which of them are its own."""
    offs = s["offs"].long()
    r = offs[:-1, None] + torch.arange(s["most"], device="cuda")
    return r.clamp(max=s["M"] - 1), (r < offs[1:, None])[..., None]


def _to_rows(s, padded):
    """[G, most, C] back to the routed rows [M, C]."""
    offs = s["offs"].long()
    i = torch.arange(s["M"], device="cuda")
    g = torch.searchsorted(offs[1:], i, right=True)
    return padded[g, i - offs[g]]


def _plain_gemm(s):
    c = s["case"]
    G, N, K = c["G"], c["N"], c["K"]
    rows, mine = _expert_rows(s)
    dt = torch.float32 if c["out"] == "f32" else torch.bfloat16
    x = s["x"][rows].float() * mine if s["x"] is not None else None
    dy = s["dy"][rows].float() * mine if s["dy"] is not None else None
    out = {}
    if "f" in c["dirs"]:
        out["y"] = _to_rows(s, torch.bmm(x, s["w"].float().view(G, N, K).transpose(1, 2))).to(dt)
    if "d" in c["dirs"]:
        out["dx"] = _to_rows(s, torch.bmm(dy, s["w"].float().view(G, N, K))).to(dt)
    if "w" in c["dirs"]:
        out["dw"] = torch.bmm(dy.transpose(1, 2), x)
    return out


def _codes(x):
    """Codes -127 .. 127 and the scale of each row."""
    amax = x.abs().amax(dim=1, keepdim=True)
    amax = torch.where(amax > 0, amax, torch.full_like(amax, 127))
    return torch.round(x * 127 / amax), amax / 127


def _plain_int8(s):
    c = s["case"]
    x = s["x"].float()
    if c["gated"]:        # in 64 bits: a value next to a border between two codes must not change sides
        gate, up = s["x"][:, :c["K"]].double(), s["x"][:, c["K"]:].double()
        x = gate / (1 + torch.exp(-gate)) * up
    q, sx = (t.float() for t in _codes(x))
    rows, mine = _expert_rows(s)
    w = s["qw"].float().view(c["G"], c["N"], c["K"]).transpose(1, 2)
    acc = torch.bmm(q[rows] * mine, w)
    y = acc * (sx[rows] * s["sw"].view(c["G"], 1, c["N"]))
    return {"y": _to_rows(s, y).to(torch.float32 if c["out"] == "f32" else torch.bfloat16)}


def _blocks(t):
    n = t.numel()
    full = torch.zeros(-(-n // 128) * 128, device=t.device, dtype=t.dtype)
    full[:n] = t
    return full.view(-1, 128)


def _pack_m(m):
    """E4M3 codes of a first moment and the scale of each 128."""
    b = _blocks(m)
    s = (b.abs().amax(dim=1) / 448).clamp_min(TINY)
    q = (b / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(-1)[: m.numel()].clone(), s


def _pack_v(v):
    """Codes of a second moment (five bits of exponent, three of mantissa, no sign; 0 is zero) and scales."""
    b = _blocks(v)
    s = (b.amax(dim=1) / TOP).clamp_min(TINY)
    bits = (b / s[:, None]).view(torch.int32)
    q = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - 96 * 8
    q = torch.where(b > 0, q.clamp(1, 255), torch.zeros_like(q)).to(torch.uint8)
    return q.reshape(-1)[: v.numel()].clone(), s


def _unpack_m(q, s):
    return (_blocks(q.view(torch.float8_e4m3fn).float()) * s[:, None]).reshape(-1)[: q.numel()]


def _unpack_v(q, s):
    c = _blocks(q.int())
    y = torch.where(c > 0, ((c + 96 * 8) << 20).view(torch.float32), torch.zeros_like(c, dtype=torch.float32))
    return (y * s[:, None]).reshape(-1)[: q.numel()]


def _plain_adamw_one(s, i):
    eight = s["case"]["bits"] == 8
    p, m, v = s["p"][i], s["m"][i], s["v"][i]
    g = s["g"][i].float() * s["scale"]
    m32 = _unpack_m(m, s["ms"][i]) if eight else m
    v32 = _unpack_v(v, s["vs"][i]) if eight else v
    m32 = s["beta1"] * m32 + (1 - s["beta1"]) * g
    v32 = s["beta2"] * v32 + (1 - s["beta2"]) * g * g
    root = torch.sqrt(v32 / (1 - s["beta2"] ** s["step"])) + s["eps"]
    p.copy_(p * (1 - s["lr"] * s["wd"]) - s["lr"] * (m32 / (1 - s["beta1"] ** s["step"])) / root)
    s["w"][i].copy_(p)
    if eight:
        for buf, scales, (q, sc) in ((m, s["ms"][i], _pack_m(m32)), (v, s["vs"][i], _pack_v(v32))):
            buf.copy_(q)
            scales.copy_(sc)
        return p, s["w"][i], _unpack_m(m, s["ms"][i]).to(torch.bfloat16), _unpack_v(v, s["vs"][i]).to(torch.bfloat16)
    m.copy_(m32)
    v.copy_(v32)
    return p, s["w"][i], m, v


def _plain_adamw(s):
    return {"tensors": [_plain_adamw_one(s, i) for i in range(len(s["p"]))]}


# ------------------------------------------------------------------------------------ the framework's
def _own_gemm(s):
    import precision_moe_expert_mx_amd as mx
    c = s["case"]
    out = {}
    if "f" in c["dirs"]:
        out["y"] = mx.bf16_grouped_gemm_fwd(s["x"], s["w"], s["offs"], c["N"], c["out"])
    if "d" in c["dirs"]:
        out["dx"] = mx.bf16_grouped_gemm_dgrad(s["dy"], s["w"], s["offs"], c["K"], c["out"])
    if "w" in c["dirs"]:
        out["dw"] = mx.bf16_grouped_gemm_wgrad(s["dy"], s["x"], s["offs"], "f32")
    return out


def _own_int8(s):
    import precision_moe_expert_mx_amd as mx
    c = s["case"]
    q, sx = mx.int8_quantize_swiglu_rowwise(s["x"]) if c["gated"] else mx.int8_quantize_rowwise(s["x"])
    return {"y": mx.int8_grouped_gemm_fwd(q, sx, s["qw"], s["sw"], s["offs"], c["N"], c["out"])}


def _own_adamw(s):
    import precision_moe_expert_mx_amd as mx
    eight = s["case"]["bits"] == 8
    if s["table"] is None:       # a program makes it once, with its tensors
        s["table"] = mx.adamw_table(s["p"], s["g"], s["m"], s["v"], weights=s["w"],
                                    exp_avg_scales=s["ms"] if eight else None,
                                    exp_avg_sq_scales=s["vs"] if eight else None)
    mx.adamw_step(s["table"], s["step"], s["lr"], s["beta1"], s["beta2"], s["eps"], s["wd"], grad_scale=s["scale"])
    if not eight:
        return {"tensors": list(zip(s["p"], s["w"], s["m"], s["v"]))}
    return {"tensors": [(s["p"][i], s["w"][i], mx.adamw_dequantize(s["m"][i], s["ms"][i], "exp_avg", "bf16"),
                         mx.adamw_dequantize(s["v"][i], s["vs"][i], "exp_avg_sq", "bf16"))
                        for i in range(len(s["p"]))]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"gemm": _own_gemm, "int8": _own_int8, "adamw": _own_adamw}[op](state)
    return {"gemm": _plain_gemm, "int8": _plain_int8, "adamw": _plain_adamw}[op](state)


# ----------------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        eight = case["bits"] == 8
        # weight read and written, its bf16 copy, the gradient, the moments read and written (8 bits: and
        # their values written in bf16)
        per = 8 + 2 + (2 if case["grad"] == "bf16" else 4) + (4 + 4 if eight else 16)
        return {"bytes": n * per, "flops": 20 * n}
    G, N, K, M = case["G"], case["N"], case["K"], case["T"] * case["top"]
    # experts that a token reaches: their weights have to be read
    hit = G * (1 - (1 - case["top"] / G) ** case["T"])
    ob = 4 if case["out"] == "f32" else 2
    if case["op"] == "int8":
        return {"bytes": int(hit * N * (K + 4) + M * K * (4 if case["gated"] else 2) + M * N * ob),
                "flops": 2 * M * N * K}
    bytes_, dirs = 0, case["dirs"]
    for d in dirs:
        bytes_ += {"f": hit * N * K * 2 + M * K * 2 + M * N * ob, "d": hit * N * K * 2 + M * N * 2 + M * K * ob,
                   "w": M * (N + K) * 2 + G * N * K * 4}[d]
    return {"bytes": int(bytes_), "flops": 2 * M * N * K * len(dirs)}


# ------------------------------------------------------------------------------------- in 64 bits
def _each_expert(s, fn, out):
    offs = s["offs"].tolist()
    for g in range(len(offs) - 1):
        if offs[g + 1] > offs[g]:
            out[offs[g]:offs[g + 1]] = fn(g, slice(offs[g], offs[g + 1]))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "adamw":
        return {"tensors": [_exact_adamw(s, i) for i in range(len(s["p"]))]}
    G, N, K, M = case["G"], case["N"], case["K"], s["M"]
    if case["op"] == "gemm":
        w = s["w"].view(G, N, K)
        out = {}
        if "f" in case["dirs"]:
            out["y"] = _each_expert(s, lambda g, r: s["x"][r].to(f64) @ w[g].to(f64).t(),
                                    torch.empty((M, N), device="cuda", dtype=f64))
        if "d" in case["dirs"]:
            out["dx"] = _each_expert(s, lambda g, r: s["dy"][r].to(f64) @ w[g].to(f64),
                                     torch.empty((M, K), device="cuda", dtype=f64))
        if "w" in case["dirs"]:
            offs = s["offs"].tolist()
            dw = torch.zeros((G, N, K), device="cuda", dtype=f64)
            for g in range(G):
                r = slice(offs[g], offs[g + 1])
                dw[g] = s["dy"][r].to(f64).t() @ s["x"][r].to(f64)
            out["dw"] = dw
        return out

    def rows(g, r):
        x = s["x"][r].to(f64)
        if case["gated"]:
            x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
        amax = x.abs().max(dim=1, keepdim=True).values
        amax[amax == 0] = 127
        codes = torch.round(127 * x / amax)
        wide = s["qw"][g * N:(g + 1) * N].to(f64)
        return codes @ wide.t() * (amax / 127) * s["sw"][g * N:(g + 1) * N].to(f64)

    return {"y": _each_expert(s, rows, torch.empty((M, N), device="cuda", dtype=f64))}


def _exact_adamw(s, i):
    f64 = torch.float64
    n, eight = s["p"][i].numel(), s["case"]["bits"] == 8

    def per_block(scales):
        return scales.to(f64).repeat_interleave(128)[:n]

    def block_max(t):
        pad = torch.zeros((n + 127) // 128 * 128, device="cuda", dtype=f64)
        pad[:n] = t.abs()
        return pad.reshape(-1, 128).max(dim=1).values

    m, v = s["m"][i], s["v"][i]
    if eight:
        m = m.view(torch.float8_e4m3fn).to(f64) * per_block(s["ms"][i])
        code = v.to(f64)
        power = torch.floor(code / 8)
        v = torch.where(code > 0, (1 + (code - 8 * power) / 8) * 2.0 ** (power - 31), 0.0) * per_block(s["vs"][i])
    g = s["g"][i].to(f64) * 0.75
    m = s["beta1"] * m.to(f64) + (1 - s["beta1"]) * g
    v = s["beta2"] * v.to(f64) + (1 - s["beta2"]) * g ** 2
    hat_m, hat_v = m / (1 - s["beta1"] ** s["step"]), v / (1 - s["beta2"] ** s["step"])
    p = s["p"][i].to(f64)
    p = p - s["lr"] * s["wd"] * p - s["lr"] * hat_m / (hat_v.sqrt() + s["eps"])
    if not eight:
        return p, p, m, v
    # nearest of four significant bits, the first moment's steps no finer than those at 2^-6
    sm = (block_max(m) / 448).clamp(min=TINY).repeat_interleave(128)[:n]
    y = m / sm
    step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    m = torch.clamp(torch.round(y / step) * step, -448, 448) * sm
    sv = (block_max(v) / TOP).clamp(min=TINY).repeat_interleave(128)[:n]
    y = v / sv
    step = 2.0 ** (torch.floor(torch.log2(y.clamp(min=2.0 ** -31))) - 3)
    y = torch.clamp(torch.round(y / step) * step, 1.125 * 2.0 ** -31, TOP)
    return p, p, m, torch.where(v > 0, y * sv, 0.0)
