"""GPU tests of the plain-operand products, the int8 quantisers and the AdamW step at the ends of what their
contract allows: offsets out of order, values near the ends of fp32, long sums and long tensors."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, host, require_gpu
from workloads import f32_to_bf16_bits, routing_offsets

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                     # half a step of fp32, relative


@pytest.mark.parametrize("G,M", [(6, 6144), (7, 6272), (49, 768)])
def test_offsets_out_of_order_list_more_tiles_than_a_small_launch_counts(G, M):
    """Every other expert claims all rows, so the list is longer than any valid offsets' and a workgroup of a small
    launch takes several of its tiles.  All experts have the same weights, so every tile computed writes the same
    values: the outputs are the product, and nothing around them is written."""
    m = require_gpu()
    N, K = 128, 64
    gen = torch.Generator(device="cuda").manual_seed(G)
    offs = torch.tensor([(g % 2) * M for g in range(G + 1)], dtype=torch.int32, device="cuda")
    x = torch.randn(M, K, device="cuda", generator=gen).bfloat16()
    w = torch.randn(N, K, device="cuda", generator=gen).bfloat16()
    y, dx, y8 = (torch.full((M * c + 4096,), 3.0, device="cuda") for c in (N, K, N))
    m.bf16_grouped_gemm_fwd(x, w.repeat(G, 1), offs, N, y=y[:M * N].view(M, N))
    dy = torch.randn(M, N, device="cuda", generator=gen).bfloat16()
    m.bf16_grouped_gemm_dgrad(dy, w.repeat(G, 1), offs, K, dx=dx[:M * K].view(M, K))
    qx, sx = m.int8_quantize_rowwise(x)
    qw, sw = m.int8_quantize_rowwise(w)
    m.int8_grouped_gemm_fwd(qx, sx, qw.repeat(G, 1), sw.repeat(G), offs, N, y=y8[:M * N].view(M, N))
    for t in (y, dx, y8):
        assert (t[-4096:] == 3.0).all()
    for got, a, b in ((y, x, w.t().contiguous()), (dx, dy, w)):
        a, b = a.double(), b.double()
        assert bool(((got[:-4096].view(M, -1).double() - a @ b).abs() <= 1e-5 * (a.abs() @ b.abs())).all())
    ref = (qx.double() @ qw.double().t().contiguous()) * sx.double()[:, None] * sw.double()
    assert bool(((y8[:-4096].view(M, N).double() - ref).abs() <= 2.0 ** -22 * ref.abs()).all())


def _swiglu_codes(y):
    """Float64 codes and scales of silu(gate) * up of bf16 bit patterns [R, 2C]."""
    g, u = np.split(oracle.bf16_bits_to_f64(y), 2, axis=1)
    with np.errstate(over="ignore"):
        return oracle.int8_quantize_rows(g / (1 + np.exp(-g)) * u)


def _check_swiglu(m, gates, ups):
    y = f32_to_bf16_bits(np.concatenate([gates, ups], axis=1).astype(np.float32))
    q, s = m.int8_quantize_swiglu_rowwise(dev(y).view(torch.bfloat16))
    rq, rs = _swiglu_codes(y)
    bad = np.flatnonzero((host(q) != rq).any(axis=1))
    assert bad.size == 0, f"rows {bad[:5]}: {int((host(q) != rq).sum())} codes differ"
    # both are a float64 value (off by a few 2^-52) rounded to fp32: at most one step apart
    np.testing.assert_allclose(host(s), rs, rtol=2.0 ** -23, atol=2.0 ** -149)


@pytest.mark.parametrize("C", [8, 264, 1408, 2048, 2056, 4104, 9000])
def test_swiglu_saturated_gates_with_large_ups(C):
    """e^-g overflows fp32, its reciprocal is subnormal, or g itself is, and an up of 1e3 to 1e38 makes an ordinary
    value of it, beside ordinary and small ones: the maximum of the row, or a code, or next to nothing."""
    m = require_gpu()
    rng = np.random.default_rng(C)
    R = 48
    gates, ups = rng.normal(0, 1, (R, C)), rng.normal(0, 1, (R, C)) * 10.0 ** rng.uniform(-9, 0, (R, 1))
    few = max(1, C // 64)
    for r in range(R):
        at = rng.choice(C, few, replace=False)
        sign = rng.choice([-1.0, 1.0], few)
        if r % 3 == 2:                               # gates near or below the smallest normal number
            gates[r, at] = sign * 10.0 ** rng.uniform(-40, -37, few)
            ups[r, at] = 10.0 ** rng.uniform(3, 38, few)
        else:                                        # saturated gates; the value at most 1e3
            g = rng.uniform(-170, -80, few)
            gates[r, at] = g
            ups[r, at] = sign * 10.0 ** np.minimum(rng.uniform(3, 38.4, few), 3 - np.log10(-g) - g / np.log(10))
    _check_swiglu(m, gates, ups)


def test_swiglu_saturated_gates_by_hand():
    m = require_gpu()
    gates = np.full((5, 8), 1.0)
    ups = np.zeros((5, 8))
    gates[0, :2], ups[0, :2] = (-90, 1), (1e32, 1e-6)
    gates[1, :2], ups[1, :2] = (-88.5, -60), (2e6, 1e-4)
    gates[2, :2], ups[2, :2] = (1, -89), (1, 9.97e37)
    gates[3, :2], ups[3, :2] = (1e-39, 1), (3e38, 0.01)
    gates[4, :2], ups[4, :2] = (-120, -87), (-3e38, 1e-20)
    _check_swiglu(m, gates, ups)


def test_quantisers_of_more_rows_than_a_launch_has_workgroups():
    m = require_gpu()
    R, C = (1 << 26) + 1001, 8
    x = torch.randint(0, 1 << 14, (R, 2 * C), device="cuda", dtype=torch.int16)      # finite magnitudes below 2
    for fn, y in ((m.int8_quantize_rowwise, x[:, :C].contiguous()), (m.int8_quantize_swiglu_rowwise, x)):
        q, s = fn(y)
        for part in (slice(0, 9), slice((1 << 26) - 9, (1 << 26) + 9), slice(R - 9, R)):
            q1, s1 = fn(y[part].contiguous())
            assert torch.equal(q[part], q1) and torch.equal(s[part], s1)
        del q, s


def test_values_of_more_moments_than_a_launch_has_workgroups():
    m = require_gpu()
    n = (1 << 36) + 5001
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 3.1 * n:
        pytest.skip("needs 213 GB of GPU memory")
    q = torch.empty(n, dtype=torch.uint8, device="cuda")
    s = torch.empty(-(-n // 128), device="cuda")
    out = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    k = 128 * 80 + n % 128
    for part, scales in ((slice(0, 128 * 9), slice(0, 9)), (slice(n - k, n), slice(-81, None))):
        q[part].random_(0, 127)                      # (no NaN codes)
        s[scales].uniform_(0.5, 2)
    for name in ("exp_avg", "exp_avg_sq"):
        m.adamw_dequantize(q, s, name, "bf16", out=out)
        for part, scales in ((slice(0, 128 * 9), slice(0, 9)), (slice(n - k, n), slice(-81, None))):
            assert torch.equal(out[part], m.adamw_dequantize(q[part].clone(), s[scales].clone(), name, "bf16"))
    del q, s, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("sizes,N,K", [([1, 0, 2], 264, 4096), ([300, 5, 700], 520, 1008), ([1500, 1, 2000], 4104, 208)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_int8_scales_whose_product_leaves_fp32(sizes, N, K, dt):
    """Scales whose product is subnormal or overflows while the output does not, and sums of zero beside them."""
    m = require_gpu()
    rng = np.random.default_rng(N)
    offs = routing_offsets(np.asarray(sizes))
    M, G = int(offs[-1]), len(sizes)
    qx, qw = rng.integers(-128, 128, (M, K)).astype(np.int8), rng.integers(-128, 128, (G * N, K)).astype(np.int8)
    qx[::3] = 0                                      # sums of zero
    for top in (-41.0, 41.0):                        # log10 of the product of the scales
        a = rng.uniform(8, 28, M)
        sx = (10.0 ** (np.sign(top) * a)).astype(np.float32)
        sw = (10.0 ** rng.uniform(0, 1, G * N) * 10.0 ** (top / 2)).astype(np.float32)
        if top > 0:
            qx[1::3], sx[1::3] = 0, 1e30             # (rows that are not zero would overflow)
            qx[2::3], sx[2::3] = 0, 1e25
        y = m.int8_grouped_gemm_fwd(dev(qx), dev(sx), dev(qw), dev(sw), dev(offs), N, dt)
        ref = oracle.int8_gemm_fwd(qx, sx, qw, sw, offs, N)
        ok = np.abs(ref) < 3e38
        rel = 2.0 ** -22 + (2.0 ** -8 if dt == "bf16" else 0)
        got = y.float().cpu().numpy().astype(np.float64)
        # below the smallest normal number an output is off by half a subnormal step of its type
        err = np.abs(got - ref)
        tiny = 2.0 ** -149 if dt == "f32" else 2.0 ** -133
        assert (err <= rel * np.abs(ref) + tiny)[ok].all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("size,eps", [(1e-20, 1e-30), (3e-19, 2.0 ** -126), (1e-22, 1e-25), (1e-12, 1e-20)])
def test_second_moment_below_the_smallest_normal_number(bits, size, eps):
    """Gradients whose squares are subnormal: the update divides by their root, not by eps alone.  The moments are
    the kernel's own fp32 operations; the update of those is off by its own 12 roundings (see the bound of
    test_gpu_adamw) and the 2 of the first moment's product with the rate."""
    m = require_gpu()
    rng = np.random.default_rng(1)
    n, lr, b1, b2 = 5000, 1e-2, 0.9, 0.95
    f = np.float32
    p0 = (0.02 * rng.standard_normal(n)).astype(f)
    g = (size * rng.standard_normal(n)).astype(f)
    p, zeros = dev(p0.copy()), lambda k, dt: torch.zeros(k, dtype=dt, device="cuda")  # noqa: E731
    kind = torch.uint8 if bits == 8 else torch.float32
    mom, sc = [zeros(n, kind) for _ in range(2)], [zeros(-(-n // 128), torch.float32) for _ in range(2)]
    table = m.adamw_table([p], [dev(g)], [mom[0]], [mom[1]], exp_avg_scales=[sc[0]] if bits == 8 else None,
                          exp_avg_sq_scales=[sc[1]] if bits == 8 else None)
    m.adamw_step(table, 1, lr, beta1=b1, beta2=b2, eps=eps, weight_decay=0.0)
    m1, v1 = (f(1 - b1) * g).astype(np.float64), (f(1 - b2) * g * g).astype(np.float64)
    if bits == 32:
        assert np.array_equal(host(mom[0]), m1.astype(f)) and np.array_equal(host(mom[1]), v1.astype(f))
    update = lr * (m1 / (1 - b1)) / (np.sqrt(v1 / (1 - b2)) + eps)
    err = np.abs(host(p).astype(np.float64) - (p0.astype(np.float64) - update))
    assert (err <= 3 * U * (np.abs(p0) + np.abs(update)) + 14 * U * np.abs(update)).all()


def test_nonfinite_second_moment_shows_in_its_values():
    """The element whose gradient was not finite has no finite moment, in its codes' values too, and stays so."""
    m = require_gpu()
    n = 600
    z = lambda k, dt=torch.float32: torch.zeros(k, dtype=dt, device="cuda")  # noqa: E731
    p, g = z(n), torch.randn(n, device="cuda")
    q, s = [z(n, torch.uint8) for _ in range(2)], [z(5) for _ in range(2)]
    g[200], g[450] = float("nan"), float("inf")
    table = m.adamw_table([p], [g], [q[0]], [q[1]], exp_avg_scales=[s[0]], exp_avg_sq_scales=[s[1]])
    m.adamw_step(table, 1, 1e-3)
    for k, name in enumerate(("exp_avg", "exp_avg_sq")):
        for dt in ("f32", "bf16"):
            v = m.adamw_dequantize(q[k], s[k], name, dt).float().cpu().numpy()
            assert not np.isfinite(v[[200, 450]]).any(), (name, dt)
            for b in (0, 2, 4):                      # the other blocks of 128
                assert np.isfinite(v[128 * b:128 * (b + 1)]).all()
    g.normal_()
    m.adamw_step(table, 2, 1e-3)
    for k, name in enumerate(("exp_avg", "exp_avg_sq")):
        v = m.adamw_dequantize(q[k], s[k], name).cpu().numpy()
        assert not np.isfinite(v[[200, 450]]).any(), name


@pytest.mark.parametrize("size", [1e-33, 1e-20, 3e-14, 1.0])
def test_8_bit_codes_of_small_moments_equal_any_fp32_implementation(size):
    """Gradients whose moments divided by their scale lie on a border between two codes or next to one: with b1 = b2 = 0
    the moments are g and g * g, as near to borders as fp32 has them."""
    m = require_gpu()
    rng = np.random.default_rng(46)
    f = np.float32
    blocks = 400
    g = np.zeros((blocks, 128), f)
    g[:, 0] = size * (1 + rng.random(blocks))
    smag, sv = (np.abs(g[:, 0]) * (f(1) / f(448))).astype(f), (g[:, 0] * g[:, 0] * (f(1) / f(1.875))).astype(f)
    smag, sv = np.maximum(smag, f(2.0 ** -126)), np.maximum(sv, f(2.0 ** -126))
    border_m = ((1 + (rng.integers(0, 8, (blocks, 64)) + 0.5) / 8) * 2.0 ** rng.integers(-6, 8, (blocks, 64))).astype(f)
    border_v = ((1 + (rng.integers(0, 8, (blocks, 63)) + 0.5) / 8) * 2.0 ** rng.integers(-30, 0, (blocks, 63)))
    g[:, 1:65] = border_m * smag[:, None] * rng.choice([-1, 1], (blocks, 64))
    g[:, 65:] = np.sqrt(border_v * sv.astype(np.float64)[:, None])
    g[:, 1:] = np.clip(g[:, 1:], -g[:, :1], g[:, :1])
    g = g.reshape(-1)
    z = lambda k, dt=torch.float32: torch.zeros(k, dtype=dt, device="cuda")  # noqa: E731
    q, s = [z(g.size, torch.uint8) for _ in range(2)], [z(blocks) for _ in range(2)]
    table = m.adamw_table([z(g.size)], [dev(g)], [q[0]], [q[1]], exp_avg_scales=[s[0]], exp_avg_sq_scales=[s[1]])
    m.adamw_step(table, 1, 1e-3, beta1=0.0, beta2=0.0)
    v = g * g
    ms = np.maximum(np.abs(g).reshape(-1, 128).max(1) * (f(1) / f(448)), f(2.0 ** -126))
    vs = np.maximum(v.reshape(-1, 128).max(1) * (f(1) / f(1.875)), f(2.0 ** -126))
    assert np.array_equal(host(s[0]), ms) and np.array_equal(host(s[1]), vs)
    mq = oracle.e4m3_encode(np.clip(g / np.repeat(ms, 128), -448, 448).astype(np.float64))
    bits = (v / np.repeat(vs, 128)).view(np.uint32)
    code = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20).astype(np.int64) - 96 * 8
    vq = np.where(v > 0, np.clip(code, 1, 255), 0).astype(np.uint8)
    for got, want in ((host(q[0]), mq), (host(q[1]), vq)):
        got, want = np.where(got == 128, 0, got), np.where(want == 128, 0, want)     # (-0 and 0)
        assert np.array_equal(got, want), int((got != want).sum())


@pytest.mark.parametrize("N", [8, 128, 264])
@pytest.mark.parametrize("G,rows", [(1, 64), (1, 65), (1, 700), (8, 512), (8, 513), (8, 3000)])
def test_narrow_layers_with_many_rows(G, N, rows):
    """Either side of the choice between the kernels, evenly routed and all rows on one expert."""
    m = require_gpu()
    K = 2048
    gen = torch.Generator(device="cuda").manual_seed(rows + N)
    x = torch.randn(rows, K, device="cuda", generator=gen).bfloat16()
    w = torch.randn(G * N, K, device="cuda", generator=gen).bfloat16()
    (qx, sx), (qw, sw) = m.int8_quantize_rowwise(x), m.int8_quantize_rowwise(w)
    even = [rows * g // G for g in range(G + 1)]
    for offs in (even, [0] * ((G + 1) // 2) + [rows] * (G + 1 - (G + 1) // 2)):
        o = torch.tensor(offs, dtype=torch.int32, device="cuda")
        y, y8 = m.bf16_grouped_gemm_fwd(x, w, o, N).double(), m.int8_grouped_gemm_fwd(qx, sx, qw, sw, o, N).double()
        for g in range(G):
            r, c = slice(offs[g], offs[g + 1]), slice(g * N, (g + 1) * N)
            a, b = x[r].double(), w[c].double().t().contiguous()
            assert bool(((y[r] - a @ b).abs() <= 1e-5 * (a.abs() @ b.abs())).all())
            ref = (qx[r].double() @ qw[c].double().t().contiguous()) * sx[r].double()[:, None] * sw[c].double()
            assert bool(((y8[r] - ref).abs() <= 2.0 ** -22 * ref.abs()).all())


@pytest.mark.parametrize("L", [8192, 32768, 65537])
@pytest.mark.parametrize("kind", ["equal", "one sign", "both signs"])
def test_long_sums(L, kind):
    """The three products of long contractions against float64: at most L / 8 roundings of 2^-24, taken fourfold for what
    the instruction loses inside its 8 products.  (Equal products go past 1e-5: their roundings all go one way.)"""
    m = require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(L)
    n, c, Lk = 16, 24, L // 8 * 8

    def make(rows, cols):
        if kind == "equal":
            return torch.full((rows, cols), 1 + 2.0 ** -7, device="cuda").bfloat16()
        t = torch.randn(rows, cols, device="cuda", generator=gen)
        return (t if kind == "both signs" else t.abs() + 0.1).bfloat16()

    def check(got, a, b):
        a, b = a.double(), b.double()
        assert bool(((got.double() - a @ b).abs() <= max(1e-5, 2.0 ** -25 * L) * (a.abs() @ b.abs())).all())

    offs = torch.tensor([0, 3, L + 3], dtype=torch.int32, device="cuda")
    dy, x = make(L + 3, n), make(L + 3, c)
    check(m.bf16_grouped_gemm_wgrad(dy, x, offs)[1], dy[3:].t().contiguous(), x[3:])
    for rows in (5, 300):
        o = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        a, w = make(rows, Lk), make(n, Lk)
        check(m.bf16_grouped_gemm_fwd(a, w, o, n), a, w.t().contiguous())
        w = make(Lk, c)
        check(m.bf16_grouped_gemm_dgrad(a, w, o, c), a, w)


def test_backward_with_weights_of_before_the_step_raises():
    """The step is an in-place change that autograd knows of, of the weights and of their bf16 copies."""
    m = require_gpu()
    z = lambda: torch.zeros(256, device="cuda")  # noqa: E731
    p, w, g = torch.ones(256, device="cuda"), torch.ones(256, dtype=torch.bfloat16, device="cuda"), torch.ones(256, device="cuda")
    table = m.adamw_table([p], [g], [z()], [z()], weights=[w])
    for saved in (p, w):
        x = torch.ones_like(saved, requires_grad=True)
        y = (x * saved).sum()                        # (saves the weight for x's gradient)
        m.adamw_step(table, 1, 1e-3)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
        (x * saved).sum().backward()                 # one that ran after the step is fine
        assert torch.equal(x.grad, saved)
    with torch.inference_mode():                     # (tensors without a version)
        p2, g2 = torch.ones(256, device="cuda"), torch.ones(256, device="cuda")
        m.adamw_step(m.adamw_table([p2], [g2], [z()], [z()]), 1, 1e-3)
    assert (p2 != 1).all()
