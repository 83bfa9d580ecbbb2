"""GPU parity of the AdamW step over many tensors against float64, its 8-bit moments, and the training run
that it closes: products, gradients, update, quantised weights."""
import numpy as np
import pytest
import torch

import oracle
import precision_moe_expert_mx_amd as mm
from gpu_util import dev, host, random_bf16, require_gpu
from workloads import f32_to_bf16_bits, routing_offsets

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                     # half a step of fp32, relative
HYPER = dict(beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


def _bound_m(m, g, b1):
    """b1 and 1 - b1 in fp32, the scaled gradient, the product and the fma: at most 5 roundings of a term."""
    return 5 * U * (np.abs(b1 * m) + np.abs((1 - b1) * g))


def _bound_p(p, m, g, v1, step, lr, h):
    """3 roundings of p (the decay factor, its product, the fma) and of the update: v's relative error
    (6 roundings) and those of v / (1 - b2^t) (2), halved by the root, the root (2: one unit in the last
    place), the sum with eps (1), the reciprocal (2), lr / (1 - b1^t) (1), two products (2): 12, and m's."""
    root = np.sqrt(v1 / (1 - h["beta2"] ** step)) + h["eps"]
    rate = lr / (1 - h["beta1"] ** step) / root
    terms = np.abs(h["beta1"] * m) + np.abs((1 - h["beta1"]) * g)
    return 3 * U * np.abs(p) + rate * (12 + 5) * U * terms


def _make(rng, n, bits, gdt):
    p = (0.02 * rng.standard_normal(n)).astype(np.float32)
    g = (1e-3 * rng.standard_normal(n)).astype(np.float32)
    if gdt == "bf16":
        g = (f32_to_bf16_bits(g).astype(np.uint32) << 16).view(np.float32)
    m = (5e-4 * rng.standard_normal(n)).astype(np.float32)
    v = ((1e-3 * rng.standard_normal(n)) ** 2).astype(np.float32)
    z = n // 3
    g[:z], m[:z // 2], v[:z // 2] = 0, 0, 0          # weights whose expert got no token
    d = {"p": dev(p), "w": torch.zeros(n, dtype=torch.bfloat16, device="cuda"), "g": dev(g)}
    if gdt == "bf16":
        d["g"] = d["g"].to(torch.bfloat16)
    if bits == 8:
        (mq, ms), (vq, vs) = oracle.adamw_pack_m(m.astype(np.float64)), oracle.adamw_pack_v(v.astype(np.float64))
        d.update(m=dev(mq), ms=dev(ms), v=dev(vq), vs=dev(vs))
        m, v = oracle.adamw_unpack_m(mq, ms), oracle.adamw_unpack_v(vq, vs)
    else:
        d.update(m=dev(m), v=dev(v))
    return d, [a.astype(np.float64) for a in (p, g, m, v)]


def _table(m, ts, bits, weights=True):
    col = lambda k: [t[k] for t in ts]  # noqa: E731
    return m.adamw_table(col("p"), col("g"), col("m"), col("v"), weights=col("w") if weights else None,
                         exp_avg_scales=col("ms") if bits == 8 else None,
                         exp_avg_sq_scales=col("vs") if bits == 8 else None)


def _check(d, before, bits, step, lr, scale, h=HYPER, weights=True):
    p0, g, m0, v0 = before
    p, m, v = oracle.adamw(p0, g, m0, v0, step, lr, h["beta1"], h["beta2"], h["eps"], h["weight_decay"], scale)
    got = host(d["p"])
    assert (np.abs(got - p) <= _bound_p(p, m0, g * scale, v, step, lr, h)).all()
    if weights:
        assert np.array_equal(host(d["w"]), f32_to_bf16_bits(got))
    bm = _bound_m(m0, g * scale, h["beta1"])
    if bits == 32:
        assert (np.abs(host(d["m"]) - m) <= bm).all()
        assert (np.abs(host(d["v"]) - v) <= 6 * U * v).all()
        return
    # codes: half a step of what was rounded, whatever side of a border fp32 put it on
    (rq, rs), (wq, ws) = oracle.adamw_pack_m(m), oracle.adamw_pack_v(v)
    np.testing.assert_allclose(host(d["ms"]), rs, rtol=1e-6)
    np.testing.assert_allclose(host(d["vs"]), ws, rtol=1e-6)
    n = m.size
    sm, sv = (np.repeat(host(d[k]).astype(np.float64), 128)[:n] for k in ("ms", "vs"))
    gm, gv = oracle.adamw_unpack_m(host(d["m"]), host(d["ms"])), oracle.adamw_unpack_v(host(d["v"]), host(d["vs"]))
    assert (np.abs(gm - m) <= np.maximum(np.abs(m) * 2.0 ** -4, sm * 2.0 ** -10) * (1 + 1e-5) + bm).all()
    assert (np.abs(gv - v) <= np.maximum(v * 2.0 ** -4 * (1 + 1e-5), sv * 1.125 * 2.0 ** -31)).all()
    assert ((gv > 0) == (v > 0)).all()
    # a value next to a border may fall on either side: 16 U wide borders, 8 to a binade, hold 1e-5 of them
    for a, b in ((host(d["m"]), rq), (host(d["v"]), wq)):
        assert (a != b).sum() <= 3 + 1e-4 * n


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gdt", ["f32", "bf16"])
def test_many_tensors(bits, gdt):
    """Lengths from none and one to several blocks, odd ones among them, in one table (two launches)."""
    m = require_gpu()
    rng = np.random.default_rng(bits)
    lengths = [0, 1, 2, 3, 4, 5, 127, 128, 129, 1000, 1023, 1024, 1025, 4096, 4097, 5000, 12345] + list(range(60, 95))
    made = [_make(rng, n, bits, gdt) for n in lengths]
    table = _table(m, [d for d, _ in made], bits)
    scale = torch.full((1,), 0.5, device="cuda")
    m.adamw_step(table, 3, 1e-3, grad_scale=scale, **HYPER)
    for (d, before), n in zip(made, lengths):
        if n:
            _check(d, before, bits, 3, 1e-3, 0.5)


@pytest.mark.parametrize("bits", [32, 8])
def test_large_tensor_and_no_copies(bits):
    m = require_gpu()
    rng = np.random.default_rng(20 + bits)
    d, before = _make(rng, 5_000_003, bits, "f32")
    m.adamw_step(_table(m, [d], bits, weights=False), 1, 3e-4, **HYPER)
    _check(d, before, bits, 1, 3e-4, 1.0, weights=False)
    assert not d["w"].any()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("hyper", [dict(beta1=0.0, beta2=0.0, eps=1e-3, weight_decay=0.0),
                                   dict(beta1=0.99, beta2=0.999, eps=1e-12, weight_decay=0.01)])
def test_hyperparameters(bits, hyper):
    m = require_gpu()
    rng = np.random.default_rng(30 + bits)
    for step, lr in ((1, 0.1), (100000, 1e-6), (2, 0.0)):
        d, before = _make(rng, 3000, bits, "f32")
        m.adamw_step(_table(m, [d], bits), step, lr, **hyper)
        _check(d, before, bits, step, lr, 1.0, hyper)


def test_moments_start_from_zero_and_run():
    """Ten steps from zero moments: 8-bit moments stay near the fp32 ones, each rounding within half a step
    of what that step computed."""
    m = require_gpu()
    rng = np.random.default_rng(40)
    n = 1000
    p = (0.02 * rng.standard_normal(n)).astype(np.float32)
    d = {"p": dev(p), "w": torch.zeros(n, dtype=torch.bfloat16, device="cuda"), "g": torch.zeros(n, device="cuda"),
         "m": torch.zeros(n, dtype=torch.uint8, device="cuda"), "v": torch.zeros(n, dtype=torch.uint8, device="cuda"),
         "ms": torch.zeros(8, device="cuda"), "vs": torch.zeros(8, device="cuda")}
    table = _table(m, [d], 8)
    for step in range(1, 11):
        g = (1e-3 * rng.standard_normal(n)).astype(np.float32)
        g[500:] *= 0 if step < 5 else 1              # moments of half the tensor stay zero for a while
        d["g"].copy_(dev(g))
        before = [host(d["p"]).astype(np.float64), g.astype(np.float64),
                  oracle.adamw_unpack_m(host(d["m"]), host(d["ms"])), oracle.adamw_unpack_v(host(d["v"]), host(d["vs"]))]
        m.adamw_step(table, step, 1e-3, **HYPER)
        _check(d, before, 8, step, 1e-3, 1.0)


def test_values_of_8_bit_moments():
    m = require_gpu()
    rng = np.random.default_rng(41)
    for n in (1, 4, 130, 1001):
        q = rng.integers(0, 256, n).astype(np.uint8)
        q[(q & 127) == 127] = 3                       # E4M3 NaN codes are never written
        s = np.exp(rng.normal(-5, 2, -(-n // 128))).astype(np.float32)
        for moment, ref in (("exp_avg", oracle.adamw_unpack_m(q, s)), ("exp_avg_sq", oracle.adamw_unpack_v(q, s))):
            for dt, rel in (("f32", U), ("bf16", U + 2.0 ** -8)):
                got = m.adamw_dequantize(dev(q), dev(s), moment, dt).float().cpu().numpy()
                assert (np.abs(got - ref) <= rel * np.abs(ref)).all(), (n, moment, dt)
    all_codes = dev(np.arange(256, dtype=np.uint8).reshape(2, 128))
    got = m.adamw_dequantize(all_codes, torch.ones(2, device="cuda"), "exp_avg_sq")
    assert got.shape == (2, 128) and np.array_equal(host(got).reshape(-1), oracle.adamw_v_values())


@pytest.mark.parametrize("bits", [32, 8])
def test_nonfinite_gradient_shows(bits):
    m = require_gpu()
    d, _ = _make(np.random.default_rng(42), 600, bits, "f32")
    d["g"][200] = float("nan")
    d["g"][450] = float("inf")
    m.adamw_step(_table(m, [d], bits), 1, 1e-3, **HYPER)
    p = host(d["p"])
    assert not np.isfinite(p[[200, 450]]).any() and np.isfinite(np.delete(p, [200, 450])).all()
    if bits == 8:
        assert np.isfinite(host(d["ms"])).tolist() == [True, False, True, False, True]
        assert np.isfinite(host(d["vs"])).tolist() == [True, False, True, False, True]


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_with_step_and_rate_on_the_device(bits):
    """One captured step, replayed with a step count, a rate and a gradient scale that change on the GPU."""
    m = require_gpu()
    rng = np.random.default_rng(43)
    d, before = _make(rng, 2000, bits, "f32")
    t, lr, c = (torch.tensor([v], device="cuda", dtype=dt) for v, dt in
                ((0, torch.int64), (0.0, torch.float32), (1.0, torch.float32)))
    table = _table(m, [d], bits)
    saved = {k: v.clone() for k, v in d.items()}
    t.fill_(1)
    m.adamw_step(table, t, lr, grad_scale=c, **HYPER)        # warm up, then start again
    torch.cuda.synchronize()
    t.fill_(0)
    for k in d:
        d[k].copy_(saved[k])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t += 1
        m.adamw_step(table, t, lr, grad_scale=c, **HYPER)
    for step, rate, scale in ((1, 1e-3, 1.0), (2, 5e-4, 0.25), (3, 1e-4, 2.0)):
        lr.fill_(rate)
        c.fill_(scale)
        if bits == 8:
            mv = [oracle.adamw_unpack_m(host(d["m"]), host(d["ms"])), oracle.adamw_unpack_v(host(d["v"]), host(d["vs"]))]
        else:
            mv = [host(d["m"]).astype(np.float64), host(d["v"]).astype(np.float64)]
        before = [host(d["p"]).astype(np.float64), before[1]] + mv
        g.replay()
        torch.cuda.synchronize()
        assert int(t) == step
        _check(d, before, bits, step, float(np.float32(rate)), scale)


def test_training_run_of_an_expert_layer():
    """Forward, dgrad and wgrad in bf16, the update with fp32 and with 8-bit moments, then the updated weights
    through the MX and the int8 forward: every output against float64 of its own inputs."""
    m = require_gpu()
    rng = np.random.default_rng(44)
    offs = routing_offsets(np.array([40, 0, 100, 3]))
    G, M, N, K = 4, 143, 256, 128
    x, w0, dy = random_bf16(rng, (M, K)), random_bf16(rng, (G * N, K), 0.05), random_bf16(rng, (M, N), 1e-2)
    o, xd, dyd = dev(offs), dev(x).view(torch.bfloat16), dev(dy).view(torch.bfloat16)
    for bits in (32, 8):
        w = dev(w0).view(torch.bfloat16).clone()
        p = w.float()
        dw = torch.empty((G, N, K), device="cuda")
        kind = torch.uint8 if bits == 8 else torch.float32
        mom = [torch.zeros((G, N, K), dtype=kind, device="cuda") for _ in range(2)]
        sc = [torch.zeros(G * N * K // 128, device="cuda") for _ in range(2)]
        table = m.adamw_table([p], [dw], [mom[0]], [mom[1]], weights=[w],
                              exp_avg_scales=[sc[0]] if bits == 8 else None,
                              exp_avg_sq_scales=[sc[1]] if bits == 8 else None)
        for step in (1, 2, 3):
            wb = host(w)
            y = m.bf16_grouped_gemm_fwd(xd, w, o, N)
            dx = m.bf16_grouped_gemm_dgrad(dyd, w, o, K)
            m.bf16_grouped_gemm_wgrad(dyd, xd, o, dw=dw)
            assert oracle.check_gemm(host(y), *oracle.dense_gemm_fwd(x, wb, offs, N), "f32")[0]
            assert oracle.check_gemm(host(dx), *oracle.dense_gemm_dgrad(dy, wb, offs, N, K), "f32")[0]
            assert oracle.check_gemm(host(dw), *oracle.dense_gemm_wgrad(dy, x, offs), "f32")[0]
            flat = lambda t: host(t).reshape(-1)  # noqa: E731
            if bits == 8:
                mv = [oracle.adamw_unpack_m(flat(mom[0]), host(sc[0])), oracle.adamw_unpack_v(flat(mom[1]), host(sc[1]))]
            else:
                mv = [flat(t).astype(np.float64) for t in mom]
            before = [flat(p).astype(np.float64), flat(dw).astype(np.float64)] + mv
            m.adamw_step(table, step, 1e-3, **HYPER)
            _check({"p": p.view(-1), "w": w.view(-1), "m": mom[0].view(-1), "v": mom[1].view(-1), "ms": sc[0],
                    "vs": sc[1]}, before, bits, step, 1e-3, 1.0)
        assert not host(dw)[1].any()                 # an expert without tokens only decays
        wb = host(w)
        qx, sx = m.mx_quantize_rowwise(xd)
        qw, sw = m.mx_quantize_rowwise(w)
        ref = oracle.mx_gemm_fwd(*oracle.mx_quantize_rowwise(x), *oracle.mx_quantize_rowwise(wb), offs, N)
        assert oracle.check_gemm(host(m.mx_grouped_gemm_fwd(qx, sx, qw, sw, o, N)), *ref, "f32")[0]
        qx, sx = m.int8_quantize_rowwise(xd)
        qw, sw = m.int8_quantize_rowwise(w)
        f = oracle.bf16_bits_to_f64
        ref = oracle.int8_gemm_fwd(*oracle.int8_quantize_rows(f(x)), *oracle.int8_quantize_rows(f(wb)), offs, N)
        y8 = host(m.int8_grouped_gemm_fwd(qx, sx, qw, sw, o, N))
        assert (np.abs(y8 - ref) <= 2.0 ** -22 * np.abs(ref)).all()


def test_table_refuses():
    m = require_gpu()
    z = lambda n=256, dt=torch.float32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    p, g, a, b = z(), z(), z(), z()
    with pytest.raises(ValueError, match="overlap"):
        m.adamw_table([p, p], [g, g], [a, z()], [b, z()])
    with pytest.raises(ValueError, match="overlap"):
        m.adamw_table([p], [p], [a], [b])
    big = z(512)
    with pytest.raises(ValueError, match="overlap"):
        m.adamw_table([big[:256], big[128:384]], [g, g], [a, z()], [b, z()])
    m.adamw_table([p, z()], [g, g], [a, z()], [b, z()])      # one gradient for two weights is fine
    with pytest.raises(ValueError, match="elements"):
        m.adamw_table([p], [z(255)], [a], [b])
    with pytest.raises(TypeError):
        m.adamw_table([p], [g], [a], [z(dt=torch.uint8)])
    with pytest.raises(ValueError, match="scales"):
        m.adamw_table([p], [g], [z(dt=torch.uint8)], [z(dt=torch.uint8)])
    with pytest.raises(ValueError, match="contiguous"):
        m.adamw_table([z(512)[::2]], [g], [a], [b])
    t = m.adamw_table([p], [g], [a], [b])
    for bad in (dict(step=0), dict(eps=0.0), dict(beta1=1.0), dict(beta2=-0.1), dict(lr=float("nan"))):
        with pytest.raises(mm.MxMoeError):
            m.adamw_step(t, **{"step": 1, "lr": 1e-3, **bad})
    with pytest.raises(mm.MxMoeError, match="aligned"):
        m.adamw_step(m.adamw_table([z(260)[1:257]], [g], [a], [b]), 1, 1e-3)
    assert not p.any()


def test_8_bit_moments_equal_any_fp32_implementation():
    """The moments' operations are rounded one by one, so a plain fp32 implementation of the formula has the
    same codes and scales bit for bit, over several steps."""
    m = require_gpu()
    rng = np.random.default_rng(45)
    n = 300_001
    d, _ = _make(rng, n, 8, "bf16")
    table = _table(m, [d], 8)
    f = np.float32
    scale = f(0.3)
    c = torch.full((1,), float(scale), device="cuda")
    mq, ms, vq, vs = (host(d[k]) for k in ("m", "ms", "v", "vs"))
    values_m = np.array([oracle.e4m3_decode(np.array([k], np.uint8))[0] for k in range(256)])
    pad = lambda a, fill=0: np.concatenate([a, np.full(-a.size % 128, fill, a.dtype)])  # noqa: E731
    spread = lambda s: np.repeat(s, 128)[:n]  # noqa: E731
    for step in (1, 2, 3):
        g = host(d["g"].float()) * scale
        m1 = f(0.9) * (values_m.astype(f)[mq] * spread(ms)) + f(1 - 0.9) * g
        v1 = f(0.95) * (oracle.adamw_v_values().astype(f)[vq] * spread(vs)) + f(1 - 0.95) * g * g
        assert m1.dtype == f and v1.dtype == f
        ms = np.maximum(np.abs(pad(m1)).reshape(-1, 128).max(1) * (f(1) / f(448)), f(2.0 ** -126))
        vs = np.maximum(pad(v1).reshape(-1, 128).max(1) * (f(1) / f(1.875)), f(2.0 ** -126))
        mq = oracle.e4m3_encode(np.clip(m1 / spread(ms), -448, 448).astype(np.float64))
        bits = (v1 / spread(vs)).view(np.uint32)
        code = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20).astype(np.int64) - 96 * 8
        vq = np.where(v1 > 0, np.clip(code, 1, 255), 0).astype(np.uint8)
        m.adamw_step(table, step, 1e-3, grad_scale=c, **HYPER)
        for k, want in (("ms", ms), ("vs", vs), ("m", mq), ("v", vq)):
            got = host(d[k])
            if k == "m":                              # -0 and 0 are the same value
                got, want = np.where(got == 128, 0, got), np.where(want == 128, 0, want)
            assert np.array_equal(got, want), (step, k, int((got != want).sum()))


def test_tensor_beyond_32_bits():
    """The last elements of a tensor of more than 2^32 elements step as they would alone."""
    m = require_gpu()
    n = (1 << 32) + 1000
    k = 128 * 9 + n % 128                         # whole blocks of 128 and the last, short one
    p = torch.full((n,), 0.5, device="cuda")
    g = torch.empty(n, device="cuda", dtype=torch.bfloat16).fill_(0.25)
    g[-k:] = torch.randn(k, device="cuda").bfloat16()
    mq, vq = (torch.zeros(n, device="cuda", dtype=torch.uint8) for _ in range(2))
    ms, vs = (torch.zeros((n + 127) // 128, device="cuda") for _ in range(2))
    tail = [t[-k:].clone() for t in (p, g, mq, vq)] + [t[-((k + 127) // 128):].clone() for t in (ms, vs)]
    for a in ((p, g, mq, vq, ms, vs), tail):
        table = m.adamw_table([a[0]], [a[1]], [a[2]], [a[3]], exp_avg_scales=[a[4]], exp_avg_sq_scales=[a[5]])
        m.adamw_step(table, 1, 1e-2)
    assert torch.equal(p[-k:], tail[0]) and torch.equal(mq[-k:], tail[2]) and torch.equal(vq[-k:], tail[3])
    out = m.adamw_dequantize(mq, ms, "exp_avg", "bf16")
    assert torch.equal(out[-k:], m.adamw_dequantize(tail[2], tail[4], "exp_avg", "bf16"))
