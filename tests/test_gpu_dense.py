"""GPU parity of the bf16 grouped GEMMs: |gpu - ref| <= 1e-5 * sum |a b| per element against float64 (bf16
outputs: plus half a bf16 ulp), at the sizes, groupings and values where a tiled kernel can go wrong."""
import numpy as np
import pytest
import torch

import oracle
import precision_moe_expert_mx_amd as mm
from gpu_util import dev, host, random_bf16, require_gpu
from workloads import make_workload, routing_offsets

pytestmark = pytest.mark.gpu


def _bf16(a):
    return dev(a).view(torch.bfloat16)


def _values(t):
    a = host(t)
    if t.dtype == torch.bfloat16:
        return (a.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return a.astype(np.float64)


def _check(got, ref, dt, what):
    ok, worst, idx = oracle.check_gemm(_values(got), *ref, dt)
    assert ok, f"{what}: worst |err| / tolerance {worst:.3g} at flat index {idx}"


def _layer(rng, sizes, N, K, w_std=0.05):
    offs = routing_offsets(np.asarray(sizes))
    M, G = int(offs[-1]), len(sizes)
    return offs, random_bf16(rng, (M, K)), random_bf16(rng, (G * N, K), w_std), random_bf16(rng, (M, N))


def _run(m, offs, x, w, dy, N, K, dt, dirs="fdw"):
    o, xd, wd, dyd = dev(offs), _bf16(x), _bf16(w), _bf16(dy)
    if "f" in dirs:
        _check(m.bf16_grouped_gemm_fwd(xd, wd, o, N, dt), oracle.dense_gemm_fwd(x, w, offs, N), dt, "fwd")
    if "d" in dirs:
        _check(m.bf16_grouped_gemm_dgrad(dyd, wd, o, K, dt), oracle.dense_gemm_dgrad(dy, w, offs, N, K), dt, "dgrad")
    if "w" in dirs:
        _check(m.bf16_grouped_gemm_wgrad(dyd, xd, o, dt), oracle.dense_gemm_wgrad(dy, x, offs), dt, "wgrad")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_tiny_workload(dt):
    m = require_gpu()
    lay = make_workload("tiny").layers[0]
    _run(m, lay.offs, lay.x, lay.w.reshape(-1, lay.K), lay.dy, lay.N, lay.K, dt)


@pytest.mark.parametrize("N,K", [(8, 8), (8, 264), (248, 72), (256, 64), (264, 136), (520, 1000), (128, 2048)])
def test_odd_sizes(N, K):
    """Columns and contractions that end inside a tile, a stage, or one 16-byte piece."""
    m = require_gpu()
    rng = np.random.default_rng(N * 1000 + K)
    _run(m, *_layer(rng, [0, 1, 7, 64, 0, 65, 129, 300], N, K), N, K, "f32")


@pytest.mark.parametrize("sizes", [[1], [2], [0, 0, 1], [1] * 40, [16, 17, 15, 32, 33], [63, 64, 65, 127, 128, 129],
                                   [255, 256, 257, 0], [1000], [3, 0, 600, 1]])
def test_group_sizes(sizes):
    m = require_gpu()
    rng = np.random.default_rng(len(sizes) + sum(sizes))
    _run(m, *_layer(rng, sizes, 320, 192), 320, 192, "bf16")


def test_single_row_long_contraction():
    m = require_gpu()
    rng = np.random.default_rng(5)
    _run(m, *_layer(rng, [1, 0, 1, 2], 264, 7168), 264, 7168, "f32", "f")
    _run(m, *_layer(rng, [1, 0, 1, 2], 7168, 264), 7168, 264, "f32", "d")
    _run(m, *_layer(rng, [5000, 3, 1], 136, 72), 136, 72, "f32", "w")


def test_no_rows():
    m = require_gpu()
    offs = torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    dy = torch.empty((0, 136), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((3 * 136, 64), dtype=torch.bfloat16, device="cuda")
    assert m.bf16_grouped_gemm_fwd(x, w, offs, 136).shape == (0, 136)
    assert m.bf16_grouped_gemm_dgrad(dy, w, offs, 64).shape == (0, 64)
    dw = torch.full((3, 136, 64), float("nan"), device="cuda")
    m.bf16_grouped_gemm_wgrad(dy, x, offs, dw=dw)
    assert not dw.cpu().numpy().any()


def test_most_experts():
    m = require_gpu()
    rng = np.random.default_rng(6)
    sizes = np.zeros(1024, np.int64)
    sizes[rng.choice(1023, 60, replace=False)] = rng.integers(1, 40, 60)
    sizes[-1] = 33
    _run(m, *_layer(rng, sizes, 72, 88), 72, 88, "f32")


def test_other_rows_do_not_leak():
    """A NaN row stays in its own outputs: neighbours in the same tile, and the experts whose contraction ends
    next to it, are as without it; rows behind the last expert's are left as they were."""
    m = require_gpu()
    rng = np.random.default_rng(7)
    N, K = 136, 72
    offs, x, w, dy = _layer(rng, [10, 3, 50, 1], N, K)
    nan = np.uint16(0x7FC0)
    row = 12                                         # last row of expert 1
    xn, dyn = x.copy(), dy.copy()
    xn[row], dyn[row] = nan, nan
    o, wd = dev(offs), _bf16(w)
    keep = np.arange(len(x)) != row
    y = _values(m.bf16_grouped_gemm_fwd(_bf16(xn), wd, o, N))
    dx = _values(m.bf16_grouped_gemm_dgrad(_bf16(dyn), wd, o, K))
    dw = _values(m.bf16_grouped_gemm_wgrad(_bf16(dyn), _bf16(xn), o))
    assert np.isnan(y[row]).all() and np.isnan(dx[row]).all() and np.isnan(dw[1]).all()
    ref = oracle.dense_gemm_fwd(x, w, offs, N)
    assert oracle.check_gemm(y[keep], ref[0][keep], ref[1][keep], "f32")[0]
    ref = oracle.dense_gemm_dgrad(dy, w, offs, N, K)
    assert oracle.check_gemm(dx[keep], ref[0][keep], ref[1][keep], "f32")[0]
    ref = oracle.dense_gemm_wgrad(dy, x, offs)
    others = [0, 2, 3]
    assert oracle.check_gemm(dw[others], ref[0][others], ref[1][others], "f32")[0]
    # weights of one expert do not reach the next
    wn = w.copy()
    wn[N:2 * N] = nan
    y = _values(m.bf16_grouped_gemm_fwd(_bf16(x), _bf16(wn), o, N))
    dx = _values(m.bf16_grouped_gemm_dgrad(_bf16(dy), _bf16(wn), o, K))
    mine = (np.arange(len(x)) >= 10) & (np.arange(len(x)) < 13)
    assert np.isnan(y[mine]).all() and np.isfinite(y[~mine]).all()
    assert np.isnan(dx[mine]).all() and np.isfinite(dx[~mine]).all()
    # routed rows end before the tensor does
    short = dev(np.array([0, 10, 13, 40, 50], np.int32))
    out = torch.full((len(x), N), 7.0, device="cuda")
    m.bf16_grouped_gemm_fwd(_bf16(x), wd, short, N, y=out)
    assert (out[50:] == 7.0).all() and torch.isfinite(out).all()


def test_infinity_reaches_its_sums():
    m = require_gpu()
    rng = np.random.default_rng(8)
    offs, x, w, _ = _layer(rng, [40], 136, 72)
    x[3, 5] = 0x7F80                                 # +inf
    w[:, 5] = 0x3F80                                 # times 1
    for dt in ("f32", "bf16"):
        y = _values(m.bf16_grouped_gemm_fwd(_bf16(x), _bf16(w), dev(offs), 136, dt))
        assert np.isposinf(y[3]).all() and np.isfinite(np.delete(y, 3, 0)).all()


@pytest.mark.parametrize("which", ["fwd", "dgrad", "wgrad"])
def test_full_size_sampled(which):
    """The 64-expert layer at full size: rows of every expert (wgrad: whole experts' columns) against float64."""
    m = require_gpu()
    lay = make_workload("dsv3_16b", ["down"]).layers[0]
    N, K, offs = lay.N, lay.K, lay.offs
    w = lay.w.reshape(-1, K)
    o, x, dy, wd = dev(offs), _bf16(lay.x), _bf16(lay.dy), _bf16(w)
    rng = np.random.default_rng(9)
    if which == "wgrad":
        dw = _values(m.bf16_grouped_gemm_wgrad(dy, x, o)[:, ::37, ::31])
        ref = oracle.dense_gemm_wgrad(np.ascontiguousarray(lay.dy[:, ::37]), np.ascontiguousarray(lay.x[:, ::31]), offs)
        assert oracle.check_gemm(dw, *ref, "f32")[0]
        return
    rows = np.unique(np.concatenate([offs[:-1][np.diff(offs) > 0], offs[1:][np.diff(offs) > 0] - 1,
                                     rng.choice(lay.M, 64, replace=False)]))
    sizes = np.histogram(rows, bins=offs)[0]
    so = routing_offsets(sizes)
    if which == "fwd":
        got = m.bf16_grouped_gemm_fwd(x, wd, o, N, "bf16")[torch.from_numpy(rows).cuda()]
        _check(got, oracle.dense_gemm_fwd(lay.x[rows], w, so, N), "bf16", "fwd")
    else:
        got = m.bf16_grouped_gemm_dgrad(dy, wd, o, K, "bf16")[torch.from_numpy(rows).cuda()]
        _check(got, oracle.dense_gemm_dgrad(lay.dy[rows], w, so, N, K), "bf16", "dgrad")


def test_three_dimensional_weights_and_given_outputs():
    m = require_gpu()
    rng = np.random.default_rng(10)
    offs, x, w, dy = _layer(rng, [5, 9], 64, 40)
    o, xd, wd = dev(offs), _bf16(x), _bf16(w)
    y = torch.empty((14, 64), device="cuda")
    assert m.bf16_grouped_gemm_fwd(xd, wd.view(2, 64, 40), o, 64, y=y) is y
    assert torch.equal(y, m.bf16_grouped_gemm_fwd(xd.view(torch.int16), wd.view(torch.int16), o, 64))


def test_repeats_and_streams_give_the_same_bits():
    m = require_gpu()
    rng = np.random.default_rng(11)
    offs, x, w, dy = _layer(rng, [100, 0, 300], 264, 520)
    o, xd, wd, dyd = dev(offs), _bf16(x), _bf16(w), _bf16(dy)
    calls = (lambda s: m.bf16_grouped_gemm_fwd(xd, wd, o, 264, stream=s),
             lambda s: m.bf16_grouped_gemm_dgrad(dyd, wd, o, 520, stream=s),
             lambda s: m.bf16_grouped_gemm_wgrad(dyd, xd, o, stream=s))
    first = [c(None) for c in calls]
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = [c(side) for c in calls]
    with torch.cuda.stream(other):                   # two streams at once
        b = [c(other) for c in calls]
    side.synchronize()
    other.synchronize()
    for f, s, t in zip(first, a, b):
        assert torch.equal(f, s) and torch.equal(f, t)


def test_captured_step_replays():
    """Forward, dgrad and wgrad in one graph, replayed on new inputs between eager calls."""
    m = require_gpu()
    rng = np.random.default_rng(12)
    N, K = 264, 136
    offs, x, w, dy = _layer(rng, [70, 1, 200], N, K)
    offs2 = np.array([0, 3, 271, 271], np.int32)
    o, xd, wd, dyd = dev(offs), _bf16(x), _bf16(w), _bf16(dy)
    y, dx = torch.empty((271, N), device="cuda"), torch.empty((271, K), device="cuda")
    dw = torch.empty((3, N, K), device="cuda")

    def step(y, dx, dw):
        m.bf16_grouped_gemm_fwd(xd, wd, o, N, y=y)
        m.bf16_grouped_gemm_dgrad(dyd, wd, o, K, dx=dx)
        m.bf16_grouped_gemm_wgrad(dyd, xd, o, dw=dw)

    step(y, dx, dw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(y, dx, dw)
    for new in (offs, offs2, offs):
        o.copy_(dev(new))
        xd.mul_(-1)
        eager = [torch.empty_like(t) for t in (y, dx, dw)]
        step(*eager)
        for t in (y, dx, dw):
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for t, e in zip((y, dx, dw), eager):
            assert torch.equal(t, e)


def test_gradients_against_differences():
    """sum(Y * dY) changes with a step in X and W as dgrad and wgrad say (float64 differences of the oracle's
    forward, which is linear in each)."""
    m = require_gpu()
    rng = np.random.default_rng(13)
    N, K = 72, 40
    offs, x, w, dy = _layer(rng, [6, 0, 11], N, K)
    f = oracle.bf16_bits_to_f64
    dx = _values(m.bf16_grouped_gemm_dgrad(_bf16(dy), _bf16(w), dev(offs), K))
    dw = _values(m.bf16_grouped_gemm_wgrad(_bf16(dy), _bf16(x), dev(offs)))
    for _ in range(5):
        ux, uw = random_bf16(rng, x.shape), random_bf16(rng, w.shape)
        slope_x = (oracle.dense_gemm_fwd(ux, w, offs, N)[0] * f(dy)).sum()
        slope_w = (oracle.dense_gemm_fwd(x, uw, offs, N)[0] * f(dy)).sum()
        # |err| <= 1e-5 of the sums of magnitudes, per element of the gradient
        bx = (oracle.dense_gemm_dgrad(dy, w, offs, N, K)[1] * np.abs(f(ux))).sum()
        bw = (oracle.dense_gemm_wgrad(dy, x, offs)[1] * np.abs(f(uw).reshape(dw.shape))).sum()
        assert abs((dx * f(ux)).sum() - slope_x) <= 1e-5 * bx
        assert abs((dw * f(uw).reshape(dw.shape)).sum() - slope_w) <= 1e-5 * bw


@pytest.mark.parametrize("sizes", [[255, 0, 257, 1000, 64, 1, 900], [129, 640, 63, 320, 1, 1700]])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_many_tiles_odd_sizes(sizes, dt):
    """Enough columns for 256 x 256 tiles: partial row tiles of every height, columns and contractions that end
    inside a tile, a stage and a 16-byte piece."""
    m = require_gpu()
    rng = np.random.default_rng(len(sizes))
    _run(m, *_layer(rng, sizes, 4104, 200), 4104, 200, dt, "f")
    _run(m, *_layer(rng, sizes, 72, 4232), 72, 4232, dt, "d")
    _run(m, *_layer(rng, [130, 0, 77], 2568, 2440), 2568, 2440, dt, "w")


def test_many_tiles_other_rows_do_not_leak():
    m = require_gpu()
    rng = np.random.default_rng(14)
    offs, x, w, dy = _layer(rng, [300, 5, 700, 256, 1000, 600], 4104, 72)
    nan = np.uint16(0x7FC0)
    row = 304                                        # last row of expert 1
    keep = np.arange(len(x)) != row
    xn = x.copy()
    xn[row] = nan
    y = _values(m.bf16_grouped_gemm_fwd(_bf16(xn), _bf16(w), dev(offs), 4104))
    ref = oracle.dense_gemm_fwd(x, w, offs, 4104)
    assert np.isnan(y[row]).all() and oracle.check_gemm(y[keep], ref[0][keep], ref[1][keep], "f32")[0]
    offs, x, w, dy = _layer(rng, [130, 77], 2568, 2440)
    xn = x.copy()
    xn[130] = nan                                    # first row of expert 1, next to the end of expert 0's contraction
    dw = _values(m.bf16_grouped_gemm_wgrad(_bf16(dy), _bf16(xn), dev(offs)))
    ref = oracle.dense_gemm_wgrad(dy, x, offs)
    assert np.isnan(dw[1]).all() and oracle.check_gemm(dw[0], ref[0][0], ref[1][0], "f32")[0]


def test_more_tiles_than_a_workgroup_lists_at_once():
    """1024 experts' weight gradients: 80 tiles per CU, two lists of 64; experts of 0 to 3 rows."""
    m = require_gpu()
    rng = np.random.default_rng(15)
    sizes = np.arange(1024) % 4
    offs = routing_offsets(sizes)
    M, N, K = int(offs[-1]), 1280, 1024
    x, dy = random_bf16(rng, (M, K)), random_bf16(rng, (M, N))
    dw = torch.full((1024, N, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    m.bf16_grouped_gemm_wgrad(_bf16(dy), _bf16(x), dev(offs), "bf16", dw=dw)
    assert torch.isfinite(dw).all() and not dw[::4].any()
    for g in (1, 2, 3, 511, 777, 1022, 1023):
        r = slice(int(offs[g]), int(offs[g + 1]))
        ref = oracle.dense_gemm_wgrad(dy[r], x[r], np.array([0, sizes[g]], np.int32))
        ok, worst, _ = oracle.check_gemm(_values(dw[g:g + 1]), *ref, "bf16")
        assert ok, (g, worst)


@pytest.mark.parametrize("bad", [[0, 50, 20, 300, 10], [-5, 10, 10, 90, 40], [100, 0, 100, 0, 100]])
def test_invalid_offsets_stay_inside_the_buffers(bad):
    """Offsets out of order or past M: the results are unspecified, but nothing outside the outputs is written."""
    m = require_gpu()
    rng = np.random.default_rng(16)
    M, N, K = 100, 264, 136
    o, x, w, dy = dev(np.array(bad, np.int32)), _bf16(random_bf16(rng, (M, K))), _bf16(random_bf16(rng, (4 * N, K))), \
        _bf16(random_bf16(rng, (M, N)))
    y, dx, dw = (torch.full((s + 4096,), 3.0, device="cuda") for s in (M * N, M * K, 4 * N * K))
    m.bf16_grouped_gemm_fwd(x, w, o, N, y=y[:M * N].view(M, N))
    m.bf16_grouped_gemm_dgrad(dy, w, o, K, dx=dx[:M * K].view(M, K))
    m.bf16_grouped_gemm_wgrad(dy, x, o, dw=dw[:4 * N * K].view(4, N, K))
    for t in (y, dx, dw):
        assert (t[-4096:] == 3.0).all()


@pytest.mark.parametrize("rows", [1, 3, 65, 300, 500])
def test_few_rows_over_many_experts(rows):
    """Serving a layer of 64 experts: any number of rows per expert, most of them none or a few."""
    m = require_gpu()
    G, N, K = 64, 2056, 2056
    gen = torch.Generator(device="cuda").manual_seed(rows)
    to = torch.randint(0, G, (rows,), device="cuda", generator=gen)
    to[rows // 2:] = torch.where(to[rows // 2:] % 4 == 0, 5, to[rows // 2:])          # (expert 5 gets more)
    offs = torch.zeros(G + 1, device="cuda", dtype=torch.int32)
    offs[1:] = torch.bincount(to, minlength=G).cumsum(0)
    x = torch.randn(rows, K, device="cuda", generator=gen).bfloat16()
    w = torch.randn(G * N, K, device="cuda", generator=gen).bfloat16()
    y = m.bf16_grouped_gemm_fwd(x, w, offs, N).double()
    o = offs.tolist()
    for g in range(G):
        if o[g + 1] > o[g]:
            a, b = x[o[g]:o[g + 1]].double(), w[g * N:(g + 1) * N].double().t().contiguous()
            assert bool(((y[o[g]:o[g + 1]] - a @ b).abs() <= 1e-5 * (a.abs() @ b.abs())).all()), g


def test_operands_and_outputs_beyond_32_bits():
    """Weights, weight gradients and activations of more than 4 GiB: the last expert's rows are right."""
    m = require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(3)
    G, N, K = 40, 8192, 8200
    w = torch.empty((G * N, K), device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    for rows in (20, 700):                       # (few rows, whole tiles)
        offs = torch.zeros(G + 1, device="cuda", dtype=torch.int32)
        offs[-1] = rows
        x = torch.randn(rows, K, device="cuda", generator=gen).bfloat16()
        dy = torch.randn(rows, N, device="cuda", generator=gen).bfloat16()
        last = w[-N:].float()
        for got, a, b in ((m.bf16_grouped_gemm_fwd(x, w, offs, N), x, last.t().contiguous()),
                          (m.bf16_grouped_gemm_dgrad(dy, w, offs, K), dy, last)):
            a, b = a[-3:].double(), b.double()
            assert bool(((got[-3:].double() - a @ b).abs() <= 1e-5 * (a.abs() @ b.abs())).all())
        dw = m.bf16_grouped_gemm_wgrad(dy, x, offs, "bf16")
        a, b = dy[:, -5:].double().t().contiguous(), x.double()
        tol = 1e-5 * (a.abs() @ b.abs())
        assert bool(((dw[-1, -5:].double() - a @ b).abs() <= tol + 2.0 ** -8 * ((a @ b).abs() + tol)).all())
        assert not bool(dw[-2].any())
        del dw
    del w
    # rows of activations past 4 GiB
    rows, N, K = 300000, 64, 8192
    x = torch.empty((rows, K), device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    w = torch.randn(2 * N, K, device="cuda", generator=gen).bfloat16()
    offs = torch.tensor([0, 1, rows], device="cuda", dtype=torch.int32)
    y = m.bf16_grouped_gemm_fwd(x, w, offs, N)
    a, b = x[-300:].double(), w[N:].double().t().contiguous()
    assert bool(((y[-300:].double() - a @ b).abs() <= 1e-5 * (a.abs() @ b.abs())).all())
