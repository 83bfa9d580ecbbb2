"""The norm on the GPU against its float64 reference: codes and 8-bit scales exactly, values within bounds counted from
the roundings of the formula."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}          # half a step of a value of the type, relative
U = 2.0 ** -24
TINY = 2.0 ** -133                                     # the smallest steps of bf16 and fp32 (bf16's counts)


def f64(t):
    return t.detach().double().cpu().numpy()


def make(R, C, xdt, rdt, wdt, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (std * torch.randn((R, C), generator=g, device="cuda")).to(DT[xdt])
    res = None if rdt is None else (2 * std * torch.randn((R, C), generator=g, device="cuda")).to(DT[rdt])
    w = (1 + 0.3 * torch.randn(C, generator=g, device="cuda")).to(DT[wdt])
    return x, res, w


def stream_of(x, res):
    return x if res is None else (x.float() + res.float()).to(res.dtype)


def check(got, ref, tol, what):
    err = np.abs(f64(got) - ref)
    assert np.isfinite(err).all() and (err <= tol).all(), f"{what}: {np.max(err / tol):.3g} of the tolerance"


# rows of every launch shape: a wave, four waves, sixteen; lengths that end inside a wave's chunk; few and many rows
SHAPES = [(1, 8), (3, 64), (5, 1112), (2, 1024), (4, 1536), (7, 2048), (600, 2056), (3, 2056), (513, 4096), (8, 7168),
          (530, 7168), (2, 8200), (1, 20480), (2, 32768)]


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("xdt,rdt,wdt,ydt", [("bf16", None, "bf16", "bf16"), ("bf16", "bf16", "f32", "f32"),
                                             ("f32", "f32", "bf16", "bf16"), ("bf16", "f32", "f32", "bf16"),
                                             ("f32", "bf16", "f32", "f32"), ("f32", None, "f32", "f32")])
def test_fwd(R, C, xdt, rdt, wdt, ydt):
    m = require_gpu()
    x, res, w = make(R, C, xdt, rdt, wdt, seed=R + C)
    got = m.rmsnorm_fwd(x, w, 1e-5, residual=res, out_dtype=ydt)
    h = stream_of(x, res)
    if res is not None:
        got, hk = got
        assert hk.dtype == res.dtype and torch.equal(hk, h)
    ref, _ = oracle.rmsnorm(f64(h), f64(w), 1e-5)
    # r rounded once, two products: three roundings, and that of the result
    check(got, ref, (4 * U + HALF[ydt]) * np.abs(ref) + TINY, "y")


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("xdt,rdt,wdt", [("bf16", "bf16", "bf16"), ("f32", None, "f32"), ("bf16", "f32", "f32")])
def test_int8(R, C, xdt, rdt, wdt):
    m = require_gpu()
    x, res, w = make(R, C, xdt, rdt, wdt, seed=R * C)
    x[R // 2] = 0
    if res is not None:
        res[R // 2] = 0
    if wdt == "bf16":
        w[::3] = 1                                     # (quotients that are ties)
    got = m.int8_quantize_rmsnorm_rowwise(x, w, 1e-5, residual=res, with_y=True)
    h = stream_of(x, res)
    q, s = oracle.rmsnorm_int8(f64(h), f64(w), 1e-5)
    assert np.array_equal(got[0].cpu().numpy(), q)
    check(got[1], s, 1.001 * U * s, "scales")          # one rounding
    if res is not None:
        assert torch.equal(got[2], h)
    y = m.rmsnorm_fwd(h, w, 1e-5)
    assert torch.equal(got[-1], y)


@pytest.mark.parametrize("R,C", [(r, c) for r, c in SHAPES if c % 32 == 0])
@pytest.mark.parametrize("xdt,rdt,wdt", [("bf16", "bf16", "bf16"), ("f32", None, "f32"), ("bf16", "f32", "f32")])
def test_mx(R, C, xdt, rdt, wdt):
    m = require_gpu()
    x, res, w = make(R, C, xdt, rdt, wdt, seed=R * C + 1)
    x[:, 32:64] *= 1e-3                                # (a block of another size)
    x[R // 2] = 0
    if res is not None:
        res[R // 2] = 0
    got = m.mx_quantize_rmsnorm_rowwise(x, w, 1e-5, residual=res, with_y=True)
    h = stream_of(x, res)
    q, s = oracle.rmsnorm_mx(f64(h), f64(w), 1e-5)
    assert np.array_equal(got[0].cpu().numpy(), q) and np.array_equal(got[1].cpu().numpy(), s)
    if res is not None:
        assert torch.equal(got[2], h)
    assert torch.equal(got[-1], m.rmsnorm_fwd(h, w, 1e-5))


def test_codes_beside_borders():
    """int8 codes where every other quotient 127 v / amax is a tie, in bf16 and in fp32 values."""
    m = require_gpu()
    C = 512
    for dt in ("bf16", "f32"):
        v = (torch.arange(C, device="cuda") % 254).float() - 126.5        # ties of amax 127
        v[0] = 127
        x = torch.stack([v, v / 4, -v]).to(DT["f32"])
        if dt == "bf16":
            x = x.to(DT["bf16"])                       # (halves of integers below 128: 8 bits)
            assert torch.equal(x[0].float(), v)
        w = torch.ones(C, device="cuda", dtype=DT[dt])
        q, s = m.int8_quantize_rmsnorm_rowwise(x, w, 1e-6)
        ref = oracle.rmsnorm_int8(f64(x), f64(w), 1e-6)
        assert np.array_equal(q.cpu().numpy(), ref[0])
        if dt == "f32":                                # one step of fp32 to either side of a tie
            for to in (0.0, 1e9):
                xn = torch.nextafter(x, torch.full_like(x, to))
                xn[:, 0] = x[:, 0]
                q, _ = m.int8_quantize_rmsnorm_rowwise(xn, w, 1e-6)
                assert np.array_equal(q.cpu().numpy(), oracle.rmsnorm_int8(f64(xn), f64(w), 1e-6)[0])


def test_magnitudes():
    """Rows of very large and very small values: the squares are summed where they fit."""
    m = require_gpu()
    for std in (1e-30, 1e-20, 1e-3, 1e15, 1e30):
        for xdt in ("bf16", "f32"):
            x, _, w = make(4, 256, xdt, None, "f32", seed=3, std=std)
            ref, _ = oracle.rmsnorm(f64(x), f64(w), 1e-6)
            check(m.rmsnorm_fwd(x, w, 1e-6, out_dtype="f32"), ref, 5 * U * np.abs(ref) + 2.0 ** -148, f"{std}")
            q, s = m.int8_quantize_rmsnorm_rowwise(x, w, 1e-6)
            rq, rs = oracle.rmsnorm_int8(f64(x), f64(w), 1e-6)
            assert np.array_equal(q.cpu().numpy(), rq)
            check(s, rs, 1.001 * U * rs + 2.0 ** -149, "scales")
            q, s = m.mx_quantize_rmsnorm_rowwise(x, w, 1e-6)
            rq, rs = oracle.rmsnorm_mx(f64(x), f64(w), 1e-6)
            assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)


def test_products_beyond_fp32():
    """h w, and g h in the backward pass, pass the largest fp32 value where the results do not."""
    m = require_gpu()
    for C in (256, 4096):
        x, _, w = make(4, C, "bf16", None, "f32", seed=4, std=1e37)
        w *= 100
        x[1] *= 1e-37
        for wk in (w, w.to(DT["bf16"])):
            q, s = m.int8_quantize_rmsnorm_rowwise(x, wk, 1e-6)
            rq, rs = oracle.rmsnorm_int8(f64(x), f64(wk), 1e-6)
            assert np.array_equal(q.cpu().numpy(), rq)
            check(s, rs, 1.001 * U * rs, "scales")
        wk = w.clone()
        wk[3] = float("inf")
        x[2, 3] = 0
        q, s = m.int8_quantize_rmsnorm_rowwise(x, wk, 1e-6)
        assert s.isnan().all() and not q.any()
        x, _, w = make(4, C, "f32", None, "f32", seed=4, std=3e36)
        dy = 20 * x / x.abs().max()                    # (a sum of products of one sign: it does pass it)
        dx, dw = m.rmsnorm_bwd(dy, x, w, 1e-6)
        args = f64(dy), f64(x), f64(w), 1e-6, None
        rx, rw = oracle.rmsnorm_bwd(*args)
        tx, tw = bwd_tolerance(*args, rx, "f32")
        check(dx, rx, tx, "dx")
        check(dw, rw, tw, "dw")


def test_rows_with_nan_or_infinity():
    m = require_gpu()
    x, _, w = make(6, 1024, "bf16", None, "bf16")
    clean = m.int8_quantize_rmsnorm_rowwise(x, w, with_y=True)
    mx = m.mx_quantize_rmsnorm_rowwise(x, w)
    x[1, 7], x[3, 900], x[4, 0] = float("nan"), float("inf"), -float("inf")
    q, s, y = m.int8_quantize_rmsnorm_rowwise(x, w, with_y=True)
    bad, good = [1, 3, 4], [0, 2, 5]
    assert torch.isnan(s[bad]).all() and not q[bad].any()
    assert y[1].isnan().all() and y[3, 900].isnan() and y[4, 0].isnan()
    for a, b in zip((q, s, y), clean):
        assert torch.equal(a[good], b[good])
    for a, b in zip(m.mx_quantize_rmsnorm_rowwise(x, w), mx):
        assert torch.equal(a[good], b[good])


def bwd_tolerance(dy, h, w, eps, dres, dx, ydt):
    """dx: the dot product's sum passes at most 32 additions in a lane, 6 over the wave and 15 over waves, with two
    roundings per term; then a dozen roundings of the two terms; the result's own.  dw: a part's rows (1 in 256 at most),
    the parts' sum (2 + 32 + 15) and three roundings per term."""
    R, C = h.shape
    r = oracle.rmsnorm(h, w, eps)[1][:, None]
    g = np.abs(dy * w)
    mean = (g * np.abs(h)).sum(axis=1, keepdims=True) / C
    tx = r * (np.abs(h) * r * r * mean * 64 * U + 12 * U * g) + 2 * U * (0 if dres is None else np.abs(dres))
    tw = (np.ceil(R / 256) + 64) * U * (np.abs(dy * h) * r).sum(axis=0)
    return tx * 1.01 + HALF[ydt] * np.abs(dx) + TINY, tw + TINY


@pytest.mark.parametrize("R,C", SHAPES + [(3000, 256), (1200, 4104)])
@pytest.mark.parametrize("hdt,wdt,dydt,with_res", [("bf16", "f32", "bf16", True), ("f32", "bf16", "bf16", True),
                                                   ("bf16", "bf16", "f32", False), ("f32", "f32", "f32", False)])
def test_bwd(R, C, hdt, wdt, dydt, with_res):
    m = require_gpu()
    h, _, w = make(R, C, hdt, None, wdt, seed=R + 2 * C)
    dy, dres, _ = make(R, C, dydt, hdt, wdt, seed=R + 3 * C)
    dres = dres if with_res else None
    dx, dw = m.rmsnorm_bwd(dy, h, w, 1e-5, dres=dres)
    assert dx.dtype == h.dtype and dw.dtype == torch.float32
    args = f64(dy), f64(h), f64(w), 1e-5, None if dres is None else f64(dres)
    rx, rw = oracle.rmsnorm_bwd(*args)
    tx, tw = bwd_tolerance(*args, rx, hdt)
    check(dx, rx, tx, "dx")
    check(dw, rw, tw, "dw")
    # again, in place, and without dw
    again, dw2 = m.rmsnorm_bwd(dy, h, w, 1e-5, dres=dres)
    assert torch.equal(again, dx) and torch.equal(dw2, dw)
    if dres is not None:
        d = dres.clone()
        out, none = m.rmsnorm_bwd(dy, h, w, 1e-5, dres=d, dx=d, need_dw=False)
        assert out is d and none is None and torch.equal(d, dx)


def test_bwd_against_differences():
    """The gradients against differences of the forward kernel itself (fp32 rows)."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(5)
    h, dy = (torch.randn((3, 16), generator=g, device="cuda") for _ in range(2))
    w = 1 + 0.3 * torch.randn(16, generator=g, device="cuda")
    dx, dw = m.rmsnorm_bwd(dy, h, w)
    loss = lambda h, w: (m.rmsnorm_fwd(h, w, out_dtype="f32").double() * dy.double()).sum().item()
    # a step of 2^-7: the third derivative's part is below 2^-14 / 6 times a number near 1, the roundings of 16 values of
    # size 4 below 16 * 4 * 2^-23 * 2^7 = 1e-3
    step = 2.0 ** -7
    for t in range(3):
        for c in range(0, 16, 5):
            d = torch.zeros_like(h)
            d[t, c] = step
            diff = (loss(h + d, w) - loss(h - d, w)) / (2 * step)
            assert abs(diff - dx[t, c].item()) < 4e-3
    for c in range(16):
        d = torch.zeros_like(w)
        d[c] = step
        assert abs((loss(h, w + d) - loss(h, w - d)) / (2 * step) - dw[c].item()) < 2e-3


def test_in_place_stream_empty_and_given_outputs():
    m = require_gpu()
    x, res, w = make(33, 1112, "bf16", "bf16", "bf16")
    y, h = m.rmsnorm_fwd(x, w, residual=res)
    r = res.clone()
    y2, h2 = m.rmsnorm_fwd(x, w, residual=r, h=r)
    assert h2 is r and torch.equal(r, h) and torch.equal(y, y2)
    out = torch.empty_like(y)
    assert m.rmsnorm_fwd(h, w, y=out) is out and torch.equal(out, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ys, hs = m.rmsnorm_fwd(x, w, residual=res, stream=side)
    dxs, dws = m.rmsnorm_bwd(y, h, w, stream=side)
    side.synchronize()
    assert torch.equal(ys, y) and torch.equal(hs, h)
    dx, dw = m.rmsnorm_bwd(y, h, w)
    assert torch.equal(dxs, dx) and torch.equal(dws, dw)
    none = x[:0]
    y0, h0 = m.rmsnorm_fwd(none, w, residual=none)
    assert y0.shape == h0.shape == (0, 1112)
    dx0, dw0 = m.rmsnorm_bwd(none, none, w, dw=torch.ones(1112, device="cuda"))
    assert dx0.shape == (0, 1112) and not dw0.any()


def test_captured():
    """Two captured graphs with a backward pass each, replayed in turn with eager work between."""
    m = require_gpu()
    sets = [make(700, 2056, "bf16", "bf16", "f32", seed=s) for s in (1, 2)]
    def step(x, res, w):
        y, h = m.rmsnorm_fwd(x, w, residual=res)
        return (y, h, *m.rmsnorm_bwd(y, h, w, dres=res))
    eager = [step(*s) for s in sets]
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*s))
        graphs.append(g)
    for _ in range(3):
        for g, out, ref in zip(graphs, outs, eager):
            for o in out:
                o.zero_()
            g.replay()
            step(*sets[0])
            torch.cuda.synchronize()
            for a, b in zip(out, ref):
                assert torch.equal(a, b)


def test_rows_beyond_32_bit_offsets():
    """A tensor of more than 2^32 bytes (and 2^31 elements): its last rows."""
    m = require_gpu()
    C = 7168
    R = (1 << 31) // C + 600
    x = torch.empty((R, C), device="cuda", dtype=torch.bfloat16)
    x[:8].normal_()
    x[8:].fill_(0.5)
    x[-520:].normal_()
    w = torch.ones(C, device="cuda", dtype=torch.bfloat16)
    y = m.rmsnorm_fwd(x, w)
    assert torch.equal(y[-520:], m.rmsnorm_fwd(x[-520:].clone(), w))
    q, s = m.int8_quantize_rmsnorm_rowwise(x, w)
    q2, s2 = m.int8_quantize_rmsnorm_rowwise(x[-520:].clone(), w)
    assert torch.equal(q[-520:], q2) and torch.equal(s[-520:], s2)
    dx, dw = m.rmsnorm_bwd(y, x, w)
    assert torch.equal(dx[-520:], m.rmsnorm_bwd(y[-520:].clone(), x[-520:].clone(), w)[0])
