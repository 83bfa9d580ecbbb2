"""Measured cases of what stands around the experts' products of a mixture-of-experts layer.

Three families, each on the shapes that such a layer meets:

* norm: root-mean-square norm of a residual stream with the addition of the last block's output, its result in
  16 or 32 bits, in 8-bit integers with a scale per row or in E4M3 with a scale per 32 elements; and its backward;
* route: the choice of each token's experts from router logits (softmax or sigmoid scores, a bias for balance,
  groups of experts, renormalised weights), the order of the chosen pairs by expert, and the logits' gradient;
* rows: tokens' rows copied to their experts' places, the weighted sum of a token's rows brought back onto the
  residual, and the backward of both.

`run` computes them in plain torch operations, or with `own` set by the library's entry points.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # serving: 8 tokens in flight before the experts' 8-bit-integer product
        {"name": "norm decode int8", "op": "norm", "dirs": "f", "T": 8, "C": 7168, "x": "bf16", "res": "bf16",
         "w": "bf16", "out": "int8"},
        # prefill before an MXFP8 product
        {"name": "norm prefill mx", "op": "norm", "dirs": "f", "T": 8192, "C": 5120, "x": "bf16", "res": "bf16",
         "w": "bf16", "out": "mx"},
        # a training step on an odd number of tokens, the residual stream in fp32
        {"name": "norm step odd", "op": "norm", "dirs": "fb", "T": 5003, "C": 1112, "x": "bf16", "res": "f32",
         "w": "f32", "out": "bf16"},
        # a training step on the tokens of one expert shard's batch: the largest
        {"name": "norm step", "op": "norm", "dirs": "fb", "T": 65536, "C": 7168, "x": "bf16", "res": "bf16",
         "w": "f32", "out": "bf16"},
        # serving the 64-expert layer: softmax scores, six experts per token
        {"name": "route decode", "op": "route", "back": False, "T": 8, "E": 64, "top": 6, "score": "softmax",
         "bias": False, "groups": 1, "keep": 1, "renorm": False, "scale": 1.0, "dt": "f32", "first": 0, "G": 64},
        # prefill of a 256-expert layer on the GPU that holds eight of them: sigmoid, bias, the best 4 of 8 groups
        {"name": "route prefill shard", "op": "route", "back": False, "T": 8192, "E": 256, "top": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "keep": 4, "renorm": True, "scale": 2.5, "dt": "f32",
         "first": 96, "G": 8},
        # a training step on an odd number of tokens and experts, logits in bf16
        {"name": "route step odd", "op": "route", "back": True, "T": 5003, "E": 7, "top": 2, "score": "softmax",
         "bias": False, "groups": 1, "keep": 1, "renorm": True, "scale": 1.0, "dt": "bf16", "first": 0, "G": 7},
        # a training step on 65536 tokens over 256 experts
        {"name": "route step", "op": "route", "back": True, "T": 65536, "E": 256, "top": 8, "score": "softmax",
         "bias": False, "groups": 1, "keep": 1, "renorm": False, "scale": 1.0, "dt": "f32", "first": 0, "G": 256},
        # serving the 64-expert layer: rows out to the experts and back
        {"name": "rows decode", "op": "rows", "dirs": "dc", "T": 8, "top": 6, "E": 64, "C": 2048, "dt": "bf16",
         "out": "bf16", "res": True},
        # prefill: tokens' rows to eight experts each
        {"name": "rows dispatch", "op": "rows", "dirs": "d", "T": 8192, "top": 8, "E": 64, "C": 7168, "dt": "bf16",
         "out": "bf16", "res": False},
        # a training step of the 64-expert layer in fp32 rows of odd length
        {"name": "rows step odd", "op": "rows", "dirs": "dcCD", "T": 5003, "top": 3, "E": 7, "C": 1112, "dt": "f32",
         "out": "f32", "res": True},
        # a training step: weighted sums of 131072 rows and their backward
        {"name": "rows combine step", "op": "rows", "dirs": "cC", "T": 16384, "top": 8, "E": 64, "C": 7168,
         "dt": "bf16", "out": "bf16", "res": True},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["norm", "route", "rows"])
    if op == "norm":
        C = _log_int(rng, 64, 16384, 8)
        out = rng.choice(["bf16", "f32", "int8", "mx"])
        if out == "mx":
            C = max(64, C // 32 * 32)
        back = out in ("bf16", "f32") and rng.random() < 0.6
        return {"op": "norm", "dirs": "fb" if back else "f", "T": _log_int(rng, 1, min(65536, 200_000_000 // C)),
                "C": C, "x": rng.choice(["bf16", "bf16", "f32"]), "res": rng.choice(["none", "bf16", "f32"]),
                "w": rng.choice(["bf16", "f32"]), "out": out}
    if op == "route":
        E = _log_int(rng, 2, 512)
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2 or g == 1])
        keep = rng.randrange(1, groups + 1)
        top = rng.randrange(1, min(10, E // groups * keep) + 1)
        G = rng.choice([E, max(1, E // 8)])
        return {"op": "route", "back": rng.random() < 0.5, "T": _log_int(rng, 1, min(65536, 16_000_000 // E)), "E": E,
                "top": top, "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "keep": keep, "renorm": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]),
                "dt": rng.choice(["f32", "bf16"]), "first": rng.randrange(0, E - G + 1), "G": G}
    C = _log_int(rng, 64, 8192, 8)
    E = _log_int(rng, 2, 256)
    top = rng.randrange(1, min(E, 8) + 1)
    return {"op": "rows", "dirs": rng.choice(["d", "dc", "cC", "dcCD"]),
            "T": _log_int(rng, 1, min(32768, 400_000_000 // (C * top))), "top": top, "E": E, "C": C,
            "dt": rng.choice(["bf16", "bf16", "f32"]), "out": rng.choice(["bf16", "f32"]), "res": rng.random() < 0.5}


# -------------------------------------------------------------------------------------------- inputs
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1013 + salt)
    return g


def _randn(shape, gen, dt="f32", std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=_DT[dt]) * std


def prepare(case, seed):
    case = dict(case)
    gen = _gen(seed, 1)
    s = {"case": case}
    T = case["T"]
    if case["op"] == "norm":
        C = case["C"]
        s["x"] = _randn((T, C), gen, case["x"])
        s["res"] = None
        if case["res"] != "none":      # a stream whose tokens differ in size, with a few large channels
            s["res"] = _randn((T, C), gen, case["res"], 2.0)
            s["res"] *= torch.exp(0.5 * _randn((T, 1), gen)).to(s["res"].dtype)
            s["res"][:, 3::509] *= 8
        s["w"] = (1 + 0.2 * _randn((C,), gen)).to(_DT[case["w"]])
        if "b" in case["dirs"]:
            s["dy"] = _randn((T, C), gen, case["out"])
            s["dres"] = _randn((T, C), gen, case["res"]) if case["res"] != "none" else None
        return s
    if case["op"] == "route":
        E = case["E"]
        s["logits"] = (_randn((T, E), gen) + 0.3 * _randn((1, E), gen)).to(_DT[case["dt"]])
        s["bias"] = 0.1 * _randn((E,), gen) if case["bias"] else None
        if case["back"]:
            s["dw"] = _randn((T, case["top"]), gen)
        return s
    E, top, C = case["E"], case["top"], case["C"]
    logits = _randn((T, E), gen) + 0.3 * _randn((1, E), gen)
    scores, ids = logits.topk(top, dim=1)
    s["weights"] = torch.softmax(scores, dim=1)
    order = torch.sort(ids.reshape(-1), stable=True).indices
    pos = torch.empty(T * top, device="cuda", dtype=torch.int32)
    pos[order] = torch.arange(T * top, device="cuda", dtype=torch.int32)
    s["pos"] = pos.view(T, top)
    if "d" in case["dirs"]:
        s["x"] = _randn((T, C), gen, case["dt"])
    if "c" in case["dirs"]:
        s["y"] = _randn((T * top, C), gen, case["dt"])
        s["res"] = _randn((T, C), gen, case["out"]) if case["res"] else None
    if "C" in case["dirs"]:
        s["dout"] = _randn((T, C), gen, case["out"])
    if "D" in case["dirs"]:
        s["dxr"] = _randn((T * top, C), gen, case["dt"])
    return s


# --------------------------------------------------------------------------------------- plain forms
def _floor_log2(v):
    """floor(log2 v) of positive numbers, exactly."""
    return torch.frexp(v)[1] - 1


def _mx_values(y):
    """Rows in 64 bits -> the values that E4M3 codes with a power of two per 32 elements stand for."""
    b = y.view(y.shape[0], -1, 32)
    amax = b.abs().amax(dim=2, keepdim=True)
    e = torch.where(amax > 0, _floor_log2(amax) - 8, torch.full_like(amax, -127, dtype=torch.int32)).clamp(-127, 127)
    z = torch.ldexp(b, -e)
    ulp = _floor_log2(z.abs().clamp_min(2.0 ** -6)) - 3
    z = torch.ldexp(torch.round(torch.ldexp(z, -ulp)), ulp).clamp(-448, 448)
    return torch.ldexp(z, e).to(torch.bfloat16).view(y.shape)


def _plain_norm(s):
    c = s["case"]
    out = {}
    h = s["x"]
    if s["res"] is not None:
        h = (s["x"].float() + s["res"].float()).to(s["res"].dtype)
        out["h"] = h
    w = s["w"].float()
    if c["out"] in _DT:
        hf = h.float()
        r = torch.rsqrt((hf * hf).mean(dim=1, keepdim=True) + EPS)
        out["y"] = (hf * r * w).to(_DT[c["out"]])
    else:           # in 64 bits: a value next to a border between two codes must not change sides
        v = h.double()
        r = 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)
        v = v * w.double()
        if c["out"] == "mx":
            out["y"] = _mx_values(v * r)
        else:
            amax = v.abs().amax(dim=1, keepdim=True)
            some = torch.where(amax > 0, amax, torch.ones_like(amax))
            scale = torch.where(amax > 0, amax * r / 127, torch.ones_like(amax)).float()
            out["y"] = torch.round(127 * v / some).float() * scale
    if "b" in c["dirs"]:
        g = s["dy"].float() * w
        dx = r * (g - hf * (r * r * (g * hf).mean(dim=1, keepdim=True)))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        out["dx"] = dx.to(h.dtype)
        out["dw"] = (s["dy"].float() * hf * r).sum(dim=0)
    return out


def _scores(c, logits):
    if c["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _plain_route(s):
    c = s["case"]
    T, E, top, groups = c["T"], c["E"], c["top"], c["groups"]
    logits = s["logits"].double()     # the order of nearly equal scores
    p = _scores(c, logits)
    choice = logits if s["bias"] is None else p + s["bias"].double()
    if groups > 1:
        part = choice.view(T, groups, E // groups)
        if s["bias"] is None:
            best = part.amax(dim=2)
        else:
            best = part.sort(dim=2, descending=True).values[:, :, :2].sum(dim=2)
        rank = best.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros((T, groups), device="cuda", dtype=torch.bool).scatter_(1, rank, True)
        choice = part.masked_fill(~kept[:, :, None], -math.inf).view(T, E)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :top]
    sel = p.gather(1, ids)
    total = sel.sum(dim=1, keepdim=True) if c["renorm"] else torch.ones_like(sel[:, :1])
    w = c["scale"] * sel / total
    out = {"ids": ids.int(), "weights": w.float()}
    # pairs by expert, those of other GPUs' experts behind the last
    local = ids.reshape(-1) - c["first"]
    mine = (local >= 0) & (local < c["G"])
    local = torch.where(mine, local, torch.full_like(local, c["G"]))
    order = local.sort(stable=True).indices
    offs = torch.zeros(c["G"] + 2, device="cuda", dtype=torch.int32)
    offs[1:] = torch.cumsum((local[None, :] == torch.arange(c["G"] + 1, device="cuda")[:, None]).sum(dim=1), dim=0)
    place = torch.arange(T * top, device="cuda")
    out["offs"] = offs[:-1]
    out["row_idx"] = torch.where(place < offs[-2], order // top, torch.full_like(order, -1)).int()
    pos = torch.empty_like(order)
    pos[order] = place
    out["pos"] = torch.where(mine, pos, torch.full_like(pos, -1)).int().view(T, top)
    if c["back"]:
        dw = s["dw"].double()
        ds = c["scale"] * dw / total
        if c["renorm"]:
            ds = ds - (dw * w).sum(dim=1, keepdim=True) / total
        if c["score"] == "sigmoid":
            dl = torch.zeros_like(p).scatter_(1, ids, ds * sel * (1 - sel))
        else:
            dl = torch.zeros_like(p).scatter_(1, ids, ds * sel) - p * (ds * sel).sum(dim=1, keepdim=True)
        out["dlogits"] = dl.to(_DT[c["dt"]])
    return out


def _plain_rows(s):
    c = s["case"]
    out = {}
    pos, w = s["pos"].long(), s["weights"]
    dt, odt = _DT[c["dt"]], _DT[c["out"]]
    rows = c["T"] * c["top"]
    if "d" in c["dirs"]:
        xr = torch.empty((rows, c["C"]), device="cuda", dtype=dt)
        xr[pos] = s["x"][:, None, :].expand(-1, c["top"], -1)
        out["xr"] = xr
    if "c" in c["dirs"]:
        o = (s["y"].float()[pos] * w[:, :, None]).sum(dim=1)
        out["out"] = (o if s["res"] is None else o + s["res"].float()).to(odt)
    if "C" in c["dirs"]:
        d = s["dout"].float()[:, None, :]
        dy = torch.empty((rows, c["C"]), device="cuda", dtype=dt)
        dy[pos] = (w[:, :, None] * d).to(dt)
        out["dy"] = dy
        out["dweights"] = (s["y"].float()[pos] * d).sum(dim=2)
    if "D" in c["dirs"]:
        out["dx"] = s["dxr"].float()[pos].sum(dim=1).to(dt)
    return out


# ------------------------------------------------------------------------------------ the framework's
def _own_norm(s):
    import precision_moe_expert_mx_amd as mx
    c = s["case"]
    out = {}
    if c["out"] in _DT:
        got = mx.rmsnorm_fwd(s["x"], s["w"], EPS, residual=s["res"], out_dtype=c["out"])
        out["y"], h = (got, s["x"]) if s["res"] is None else got
    else:
        quantize = mx.int8_quantize_rmsnorm_rowwise if c["out"] == "int8" else mx.mx_quantize_rmsnorm_rowwise
        q, scale, *rest = quantize(s["x"], s["w"], EPS, residual=s["res"])
        h = rest[0] if rest else None
        if c["out"] == "int8":
            out["y"] = q * scale[:, None]
        else:
            power = (scale.int() << 23).view(torch.float32).to(torch.bfloat16)
            q = q.view(torch.float8_e4m3fn).to(torch.bfloat16).view(c["T"], -1, 32)
            out["y"] = (q * power[:, :, None]).view(c["T"], c["C"])
    if s["res"] is not None:
        out["h"] = h
    if "b" in c["dirs"]:
        out["dx"], out["dw"] = mx.rmsnorm_bwd(s["dy"], h, s["w"], EPS, dres=s["dres"])
    return out


def _own_route(s):
    import precision_moe_expert_mx_amd as mx
    c = s["case"]
    how = {"score": c["score"], "renormalize": c["renorm"], "scale": c["scale"]}
    ids, w, offs, row_idx, pos = mx.moe_route_sort(
        s["logits"], c["top"], c["G"], c["first"], bias=s["bias"], groups=c["groups"], keep_groups=c["keep"],
        group_top=1 if s["bias"] is None else 2, **how)
    out = {"ids": ids, "weights": w, "offs": offs, "row_idx": row_idx, "pos": pos}
    if c["back"]:
        out["dlogits"] = mx.moe_route_bwd(s["dw"], ids, s["logits"], **how)
    return out


def _own_rows(s):
    import precision_moe_expert_mx_amd as mx
    c = s["case"]
    out = {}
    if "d" in c["dirs"]:
        out["xr"] = mx.moe_dispatch(s["x"], s["pos"])
    if "c" in c["dirs"]:
        out["out"] = mx.moe_combine_fwd(s["y"], s["pos"], s["weights"], residual=s["res"], out_dtype=c["out"])
    if "C" in c["dirs"]:
        out["dy"], out["dweights"] = mx.moe_combine_bwd(s["dout"], s["pos"], s["weights"], s["y"])
    if "D" in c["dirs"]:
        out["dx"] = mx.moe_combine_fwd(s["dxr"], s["pos"], out_dtype=c["dt"])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "route": _own_route, "rows": _own_rows}[op](state)
    return {"norm": _plain_norm, "route": _plain_route, "rows": _plain_rows}[op](state)


# ----------------------------------------------------------------------------------------------- work
def work(case):
    size = {"bf16": 2, "f32": 4, "none": 0, "int8": 1, "mx": 1 + 1 / 32}
    T = case["T"]
    if case["op"] == "norm":
        C = case["C"]
        n = T * C
        res = size[case["res"]]
        per = size[case["x"]] + 2 * res + size[case["out"]]
        flops = 6 * n
        if "b" in case["dirs"]:      # the stream after the addition, the result's gradient and the stream's
            h = res or size[case["x"]]
            per += size[case["out"]] + h + res + h
            flops += 12 * n
        return {"bytes": int(n * per + C * (size[case["w"]] + (4 if "b" in case["dirs"] else 0))), "flops": flops}
    if case["op"] == "route":
        E, P = case["E"], T * case["top"]
        bytes_ = T * E * size[case["dt"]] + P * 16 + 4 * (case["G"] + 1) + (4 * E if case["bias"] else 0)
        flops = T * E * 8
        if case["back"]:             # only a softmax over all experts needs every logit again
            again = case["score"] == "softmax" and not case["renorm"]
            bytes_ += T * E * size[case["dt"]] * (2 if again else 1) + P * 8
            flops += T * E * 4
        return {"bytes": bytes_, "flops": flops}
    C, P, dt, out = case["C"], T * case["top"], size[case["dt"]], size[case["out"]]
    bytes_ = flops = 0
    for d in case["dirs"]:
        bytes_ += {"d": (T + P) * C * dt + 4 * P,
                   "c": P * C * dt + T * C * out * (2 if case["res"] else 1) + 8 * P,
                   "C": 2 * P * C * dt + T * C * out + 12 * P,
                   "D": (P + T) * C * dt + 4 * P}[d]
        flops += {"d": 0, "c": 2 * P * C, "C": 3 * P * C, "D": P * C}[d]
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "rows": _exact_rows}[case["op"]](s)


def _exact_norm(s):
    f64 = torch.float64
    c = s["case"]
    T, C = s["x"].shape
    w = s["w"].to(f64)
    out = {}
    if s["res"] is not None:
        out["h"] = torch.empty((T, C), device="cuda", dtype=f64)
    out["y"] = torch.empty((T, C), device="cuda", dtype=f64)
    if "b" in c["dirs"]:
        out["dx"] = torch.empty((T, C), device="cuda", dtype=f64)
        out["dw"] = torch.zeros(C, device="cuda", dtype=f64)
    step = max(1, (1 << 25) // C)
    for t in range(0, T, step):          # some rows at a time
        rows = slice(t, min(T, t + step))
        stream = s["x"][rows].to(f64)
        if s["res"] is not None:
            out["h"][rows] = stream + s["res"][rows].to(f64)
            # the stream is held in its own type, and that is what is normalised
            stream = out["h"][rows].float().to(s["res"].dtype).to(f64)
        rms = torch.sqrt(torch.linalg.vector_norm(stream, dim=1, keepdim=True) ** 2 / C + EPS)
        unit = stream / rms
        if c["out"] == "int8":
            big = torch.linalg.vector_norm(stream * w, ord=math.inf, dim=1, keepdim=True)
            codes = torch.round(127 * (stream * w) / torch.where(big == 0, torch.ones_like(big), big))
            out["y"][rows] = codes * (big / rms / 127)
        elif c["out"] == "mx":
            y = (unit * w).reshape(-1, 32)
            big = torch.linalg.vector_norm(y, ord=math.inf, dim=1, keepdim=True).clamp(min=2.0 ** -119)
            scale = 2.0 ** (torch.floor(torch.log2(big)) - 8)
            z = y / scale
            grid = 2.0 ** (torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
            out["y"][rows] = (torch.round(z / grid) * grid).clamp(-448, 448).mul(scale).reshape(-1, C)
        else:
            out["y"][rows] = unit * w
        if "b" in c["dirs"]:
            dy = s["dy"][rows].to(f64)
            du = dy * w
            dx = (du - unit * torch.linalg.vecdot(du, unit)[:, None] / C) / rms
            out["dx"][rows] = dx if s["dres"] is None else dx + s["dres"][rows].to(f64)
            out["dw"] += torch.linalg.vecdot(dy, unit, dim=0)
    return out


def _exact_route(s):
    c = s["case"]
    T, E, top, groups = c["T"], c["E"], c["top"], c["groups"]
    x = s["logits"].double().cpu().numpy()
    if c["score"] == "sigmoid":
        p = np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
    else:
        p = np.exp(x - np.logaddexp.reduce(x, axis=1, keepdims=True))
    rank = x if s["bias"] is None else p + s["bias"].double().cpu().numpy()
    if groups > 1:
        high = np.sort(rank.reshape(T, groups, -1), axis=2)
        high = high[:, :, -1] if s["bias"] is None else high[:, :, -2:].sum(axis=2)
        out_of = np.argsort(-high, axis=1, kind="stable")[:, c["keep"]:]
        allowed = np.ones((T, groups), dtype=bool)
        np.put_along_axis(allowed, out_of, False, axis=1)
        rank = np.where(np.repeat(allowed, E // groups, axis=1), rank, -np.inf)
    ids = np.argsort(-rank, axis=1, kind="stable")[:, :top]
    chosen = np.take_along_axis(p, ids, axis=1)
    norm = chosen.sum(axis=1, keepdims=True) if c["renorm"] else 1.0
    out = {"ids": None, "weights": torch.from_numpy(c["scale"] * chosen / norm).cuda(), "offs": None, "row_idx": None,
           "pos": None}
    if c["back"]:
        dw = s["dw"].double().cpu().numpy() * c["scale"]
        # d w_k / d s_j = (delta_kj - w_k / scale) / norm where the weights are renormalised, delta_kj where not
        ds = (dw - (dw * chosen / norm).sum(axis=1, keepdims=True)) / norm if c["renorm"] else dw
        full = np.zeros_like(p)
        np.put_along_axis(full, ids, ds, axis=1)
        slope = p * (1 - p) * full if c["score"] == "sigmoid" else p * (full - (p * full).sum(axis=1, keepdims=True))
        out["dlogits"] = torch.from_numpy(slope).cuda()
    return out


def _exact_rows(s):
    f64 = torch.float64
    c = s["case"]
    T, top, C = c["T"], c["top"], c["C"]
    rows = T * top
    out = {}
    source = torch.empty(rows, device="cuda", dtype=torch.long)          # the pair of each row
    source[s["pos"].reshape(-1).long()] = torch.arange(rows, device="cuda")
    w = s["weights"].to(f64)
    if "d" in c["dirs"]:
        out["xr"] = s["x"].to(f64)[source // top]
    if "c" in c["dirs"]:
        o = torch.zeros((T, C), device="cuda", dtype=f64) if s["res"] is None else s["res"].to(f64)
        for k in range(top):
            o += w[:, k, None] * s["y"][s["pos"][:, k].long()].to(f64)
        out["out"] = o
    if "C" in c["dirs"]:
        dout = s["dout"].to(f64)
        out["dy"] = dout[source // top] * w.reshape(-1)[source][:, None]
        out["dweights"] = torch.stack([torch.linalg.vecdot(s["y"][s["pos"][:, k].long()].to(f64), dout)
                                       for k in range(top)], dim=1)
    if "D" in c["dirs"]:
        dx = torch.zeros((T, C), device="cuda", dtype=f64)
        for k in range(top):
            dx += s["dxr"][s["pos"][:, k].long()].to(f64)
        out["dx"] = dx
    return out
