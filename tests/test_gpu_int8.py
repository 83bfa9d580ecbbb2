"""GPU parity of the 8-bit-integer quantisers (bit-exact against float64) and grouped GEMM (exact integer
sums: |err| <= 2^-22 |y|, plus half a bf16 ulp for bf16 outputs)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, host, random_bf16, require_gpu
from workloads import make_workload, routing_offsets

pytestmark = pytest.mark.gpu

# (float)sum, sx * sw and their product round once each: 3 * 2^-24 (1 + small) < 2^-22; bf16 once more
REL = {"f32": 2.0 ** -22, "bf16": 2.0 ** -22 + 2.0 ** -8}


def _bf16(a):
    return dev(a).view(torch.bfloat16)


def _values(t):
    return t.float().cpu().numpy().astype(np.float64)


def _swiglu(y):
    g, u = np.split(oracle.bf16_bits_to_f64(y), 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def _same(q, s, ref):
    rq, rs = ref
    bad = np.flatnonzero((host(q) != rq).any(axis=1) | (host(s) != rs))
    assert bad.size == 0, f"rows {bad[:5]}: {int((host(q) != rq).sum())} codes differ"


@pytest.mark.parametrize("R,C", [(1, 8), (3, 16), (5, 512), (2, 520), (7, 1408), (33, 2048), (4, 2056), (3, 4096),
                                 (2, 4104), (5, 7168), (2, 8192), (3, 8200), (2, 20000)])
def test_rowwise_exact(R, C):
    m = require_gpu()
    rng = np.random.default_rng(R * 100 + C)
    x = random_bf16(rng, (R, C), outlier_frac=0.002)
    _same(*m.int8_quantize_rowwise(_bf16(x)), oracle.int8_quantize_rows(oracle.bf16_bits_to_f64(x)))


def test_rowwise_every_magnitude_and_tie():
    """Every finite bf16 magnitude as a row's maximum, beside values at ratios where the quotient is a tie."""
    m = require_gpu()
    mag = np.arange(1, 0x7F80, dtype=np.uint16)
    rng = np.random.default_rng(1)
    x = np.zeros((mag.size, 32), np.uint16)
    x[:, 0] = mag
    # smaller magnitudes: the same significand one to seven binades down, others at random; random signs
    for k in range(1, 8):
        x[:, k] = np.where(mag >= 128 * k, mag - 128 * k, 0)
    x[:, 8:] = (mag[:, None] * rng.random((mag.size, 24))).astype(np.uint16)
    x |= (rng.integers(0, 2, x.shape) << 15).astype(np.uint16)
    _same(*m.int8_quantize_rowwise(_bf16(x)), oracle.int8_quantize_rows(oracle.bf16_bits_to_f64(x)))


def test_rowwise_zero_and_nonfinite_rows():
    m = require_gpu()
    x = np.zeros((4, 64), np.uint16)
    x[1, 3], x[2, 5], x[3, 7] = 0x7F80, 0x7FC0, 0x8000     # inf, NaN, -0
    for q, s in (m.int8_quantize_rowwise(_bf16(x)), m.int8_quantize_swiglu_rowwise(_bf16(np.concatenate([x, x], 1)))):
        s = host(s)
        assert not host(q).any() and s[0] == 1 and s[3] == 1 and not np.isfinite(s[1:3]).any()


@pytest.mark.parametrize("R,C", [(1, 8), (5, 16), (3, 512), (21, 1408), (64, 2048), (9, 2056), (5, 4104), (3, 8192),
                                 (2, 9000)])
def test_swiglu_rowwise_exact(R, C):
    m = require_gpu()
    rng = np.random.default_rng(R * 100 + C + 1)
    y = random_bf16(rng, (R, 2 * C), std=2.0, outlier_frac=0.002, outlier_mult=20.0)
    _same(*m.int8_quantize_swiglu_rowwise(_bf16(y)), oracle.int8_quantize_rows(_swiglu(y)))


def test_swiglu_rowwise_extremes():
    """Saturated gates, rows whose products are all tiny (beyond fp32 in places), zeros, and one large value."""
    m = require_gpu()
    rng = np.random.default_rng(3)
    C = 256
    y = oracle.bf16_bits_to_f64(random_bf16(rng, (8, 2 * C)))
    y[0, :C] = -90.0                                  # e^-g overflows fp32
    y[1, :C] *= 30
    y[2] = 0
    y[3, :C] *= 1e-20
    y[3, C:] *= 1e-15
    y[4, :C] = 0
    y[5, 3], y[5, C + 3] = 1e4, -3e5
    y[6, :C] = np.abs(y[6, :C]) * -50
    y[7, :C], y[7, C:] = 1e-38, 1e-10
    from workloads import f32_to_bf16_bits
    y = f32_to_bf16_bits(y.astype(np.float32))
    q, s = m.int8_quantize_swiglu_rowwise(_bf16(y))
    rq, rs = oracle.int8_quantize_rows(_swiglu(y))
    assert np.array_equal(host(q), rq)
    np.testing.assert_allclose(host(s), rs, rtol=2.0 ** -23, atol=2.0 ** -149)


def test_swiglu_rowwise_many_values_next_to_borders():
    """A million values: whatever falls next to a border between two codes has to be on float64's side."""
    m = require_gpu()
    rng = np.random.default_rng(4)
    y = random_bf16(rng, (512, 4096), std=1.5)
    _same(*m.int8_quantize_swiglu_rowwise(_bf16(y)), oracle.int8_quantize_rows(_swiglu(y)))


def _gemm(m, rng, sizes, N, K, dt, lo=-127):
    offs = routing_offsets(np.asarray(sizes))
    M, G = int(offs[-1]), len(sizes)
    qx, qw = rng.integers(lo, 128, (M, K)).astype(np.int8), rng.integers(lo, 128, (G * N, K)).astype(np.int8)
    sx, sw = np.exp(rng.normal(0, 1, M)).astype(np.float32), np.exp(rng.normal(0, 1, G * N)).astype(np.float32)
    y = m.int8_grouped_gemm_fwd(dev(qx), dev(sx), dev(qw), dev(sw), dev(offs), N, dt)
    ref = oracle.int8_gemm_fwd(qx, sx, qw, sw, offs, N)
    err = np.abs(_values(y) - ref)
    assert (err <= REL[dt] * np.abs(ref)).all(), float((err / np.maximum(np.abs(ref), 1e-30)).max())


@pytest.mark.parametrize("N,K", [(8, 16), (8, 272), (248, 80), (256, 128), (264, 144), (520, 1008), (128, 4096)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gemm_odd_sizes(N, K, dt):
    _gemm(require_gpu(), np.random.default_rng(N + K), [0, 1, 7, 64, 0, 65, 129, 300], N, K, dt)


@pytest.mark.parametrize("sizes", [[1], [0, 0, 1], [1] * 40, [16, 17, 15, 32, 33], [63, 64, 65, 127, 128, 129],
                                   [255, 256, 257, 0], [1000]])
def test_gemm_group_sizes(sizes):
    _gemm(require_gpu(), np.random.default_rng(sum(sizes)), sizes, 328, 208, "f32")


def test_gemm_longest_sum():
    """Every code -128 at the longest contraction: the int32 sum reaches 2^31 - 2^18 and is exact."""
    m = require_gpu()
    K = 131072 - 16
    qx = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    qw = torch.full((16, K), -128, dtype=torch.int8, device="cuda")
    qw[3] = 127
    one = torch.ones(16, device="cuda")
    y = m.int8_grouped_gemm_fwd(qx, one[:2], qw, one, dev(np.array([0, 1, 2], np.int32)), 8)
    ref = np.full((2, 8), 16384.0 * K)
    ref[0, 3] = -128.0 * 127 * K
    assert (np.abs(_values(y) - ref) <= REL["f32"] * np.abs(ref)).all()


def test_gemm_no_rows_and_rows_behind():
    m = require_gpu()
    qw, sw = torch.ones((2 * 64, 32), dtype=torch.int8, device="cuda"), torch.ones(128, device="cuda")
    qx, sx = torch.ones((6, 32), dtype=torch.int8, device="cuda"), torch.ones(6, device="cuda")
    offs = dev(np.array([0, 2, 4], np.int32))
    assert m.int8_grouped_gemm_fwd(qx[:0], sx[:0], qw, sw, offs * 0, 64).shape == (0, 64)
    y = torch.full((6, 64), 5.0, device="cuda")
    m.int8_grouped_gemm_fwd(qx, sx, qw, sw, offs, 64, y=y)
    assert (y[:4] == 32).all() and (y[4:] == 5).all()


def test_nonfinite_token_shows():
    m = require_gpu()
    x = torch.ones((3, 32), dtype=torch.bfloat16, device="cuda")
    x[1, 4] = float("nan")
    q, s = m.int8_quantize_rowwise(x)
    w, sw = torch.ones((8, 32), dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda")
    y = m.int8_grouped_gemm_fwd(q, s, w, sw, dev(np.array([0, 3], np.int32)), 8)
    assert not torch.isfinite(y[1]).any() and torch.isfinite(y[0]).all() and torch.isfinite(y[2]).all()


def test_expert_mlp_in_8_bits():
    """tokens -> gate and up -> SwiGLU -> down, as a server runs it: every step against float64 of its own
    inputs, then once more captured in a graph."""
    m = require_gpu()
    lay = make_workload("tiny").layers[0]
    G, M, N, K, offs = lay.G, lay.M, lay.N, lay.K, lay.offs
    H = N // 2
    rng = np.random.default_rng(6)
    down = random_bf16(rng, (G * K, H), 0.05)
    o, x = dev(offs), _bf16(lay.x)
    qw, sw = m.int8_quantize_rowwise(_bf16(lay.w.reshape(-1, K)))
    qd, sd = m.int8_quantize_rowwise(_bf16(down))

    def mlp():
        qx, sx = m.int8_quantize_rowwise(x)
        y = m.int8_grouped_gemm_fwd(qx, sx, qw, sw, o, N, "bf16")
        qh, sh = m.int8_quantize_swiglu_rowwise(y)
        return qx, sx, y, qh, sh, m.int8_grouped_gemm_fwd(qh, sh, qd, sd, o, K, "bf16")

    qx, sx, y, qh, sh, out = mlp()
    _same(qx, sx, oracle.int8_quantize_rows(oracle.bf16_bits_to_f64(lay.x)))
    ref = oracle.int8_gemm_fwd(host(qx), host(sx), host(qw), host(sw), offs, N)
    assert (np.abs(_values(y) - ref) <= REL["bf16"] * np.abs(ref)).all()
    _same(qh, sh, oracle.int8_quantize_rows(_swiglu(host(y))))
    ref = oracle.int8_gemm_fwd(host(qh), host(sh), host(qd), host(sd), offs, K)
    assert (np.abs(_values(out) - ref) <= REL["bf16"] * np.abs(ref)).all()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = mlp()
    for k in range(3):
        x.mul_(-1)
        eager = mlp()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b), k


def test_gemm_many_tiles_odd_sizes():
    """Enough columns for 256 x 256 tiles, with partial rows, columns and contractions; and few rows spread over
    many columns."""
    m = require_gpu()
    rng = np.random.default_rng(7)
    for sizes in ([255, 0, 257, 1000, 64, 1, 900], [129, 640, 63, 320, 1, 1700]):
        for dt in ("f32", "bf16"):
            _gemm(m, rng, sizes, 4104, 208, dt, lo=-128)
    _gemm(m, rng, [1, 0, 33, 2, 0, 20], 4104, 1040, "f32", lo=-128)


@pytest.mark.parametrize("rows", [1, 7, 70, 300, 500])
def test_gemm_few_rows_over_many_experts(rows):
    """64 experts and a long contraction, most experts with none or a few rows.  Sums below 2^53 are exact in
    float64, and an output is off by at most the roundings of the sum, of the scales' product and of the result:
    2^-24 each, and less than 2^-22 together."""
    m = require_gpu()
    G, N, K = 64, 2056, 4112
    gen = torch.Generator(device="cuda").manual_seed(rows)
    to = torch.randint(0, G, (rows,), device="cuda", generator=gen)
    offs = torch.zeros(G + 1, device="cuda", dtype=torch.int32)
    offs[1:] = torch.bincount(to, minlength=G).cumsum(0)
    qx = torch.randint(-128, 128, (rows, K), device="cuda", generator=gen, dtype=torch.int8)
    qw = torch.randint(-128, 128, (G * N, K), device="cuda", generator=gen, dtype=torch.int8)
    sx = torch.rand(rows, device="cuda", generator=gen) + 0.5
    sw = torch.rand(G * N, device="cuda", generator=gen) + 0.5
    y = m.int8_grouped_gemm_fwd(qx, sx, qw, sw, offs, N).double()
    o = offs.tolist()
    for g in range(G):
        if o[g + 1] > o[g]:
            r, c = slice(o[g], o[g + 1]), slice(g * N, (g + 1) * N)
            ref = (qx[r].double() @ qw[c].double().t().contiguous()) * sx[r].double()[:, None] * sw[c].double()
            assert bool(((y[r] - ref).abs() <= 2.0 ** -22 * ref.abs()).all()), g


def test_rowwise_beyond_32_bits():
    """The last rows of a tensor of more than 2^32 elements have the codes that they have alone."""
    m = require_gpu()
    R, C = 530000, 8208
    x = torch.empty((R, C), device="cuda", dtype=torch.bfloat16).normal_()
    q, s = m.int8_quantize_rowwise(x)
    q1, s1 = m.int8_quantize_rowwise(x[-7:].clone())
    assert torch.equal(q[-7:], q1) and torch.equal(s[-7:], s1)
    q, s = m.int8_quantize_swiglu_rowwise(x)
    q1, s1 = m.int8_quantize_swiglu_rowwise(x[-7:].clone())
    assert torch.equal(q[-7:], q1) and torch.equal(s[-7:], s1)
