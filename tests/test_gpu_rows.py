"""Rows out and back on the GPU: dispatch exactly, sums and gradients against the float64 reference within bounds counted
from the roundings, and a whole layer through every entry point around its products."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24
TINY = 2.0 ** -133


def f64(t):
    return t.detach().double().cpu().numpy()


def places(T, top, M, seed, drop=0.2):
    """A pos [T, top] of distinct rows below M, with pairs that have none (of several kinds)."""
    rng = np.random.default_rng(seed)
    pos = np.full(T * top, -1, np.int32)
    n = min(M, T * top)
    pos[rng.permutation(T * top)[:n]] = rng.permutation(M)[:n]
    gone = rng.random(T * top) < drop
    pos[gone] = rng.choice([-1, -2 ** 31, M, 2 ** 31 - 1], gone.sum())
    if T > 2:
        pos.reshape(T, top)[T // 2] = -1               # a token with no row at all
    return torch.from_numpy(pos.reshape(T, top)).cuda()


SHAPES = [(1, 1, 8), (3, 2, 64), (8, 6, 2048), (65, 3, 1112), (5, 64, 72), (40, 8, 7168), (2, 9, 16384), (129, 1, 520),
          (300, 4, 24)]


@pytest.mark.parametrize("T,top,C", SHAPES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32, torch.int8, torch.uint8])
def test_dispatch(T, top, C, dt):
    m = require_gpu()
    M = T * top + 3
    pos = places(T, top, M, T + C)
    x = torch.randint(-100, 100, (T, C), device="cuda").to(dt)
    ref = torch.full((M, C), 77, device="cuda").to(dt)
    xr = ref.clone()
    here = ((pos >= 0) & (pos < M)).cpu()
    t, k = here.nonzero(as_tuple=True)
    ref[pos.cpu()[t, k].long().cuda()] = x[t.cuda()]
    assert m.moe_dispatch(x, pos, xr=xr) is xr and torch.equal(xr, ref)
    for shape in ((T,), (T, 1), (T, 8), (T, 45)):
        for sdt in (torch.float32, torch.uint8):
            s = torch.randint(0, 200, shape, device="cuda").to(sdt)
            sref = torch.full((M, *shape[1:]), 99, device="cuda").to(sdt)
            xr.fill_(77)
            sr = sref.clone()
            sref[pos.cpu()[t, k].long().cuda()] = s[t.cuda()]
            got = m.moe_dispatch(x, pos, s, xr=xr, sr=sr)
            assert torch.equal(got[0], ref) and torch.equal(got[1], sref)


@pytest.mark.parametrize("T,top,C", SHAPES)
@pytest.mark.parametrize("ydt,rdt,odt,weighted", [("bf16", "bf16", "bf16", True), ("f32", None, "f32", True),
                                                  ("bf16", "f32", "f32", False), ("f32", "bf16", "bf16", True),
                                                  ("bf16", None, "bf16", False)])
def test_combine(T, top, C, ydt, rdt, odt, weighted):
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(T * C)
    M = max(1, T * top - 2)
    pos = places(T, top, M, T + 2 * C)
    y = torch.randn((M, C), generator=g, device="cuda").to(DT[ydt])
    res = None if rdt is None else torch.randn((T, C), generator=g, device="cuda").to(DT[rdt])
    w = torch.randn((T, top), generator=g, device="cuda") if weighted else None
    out = m.moe_combine_fwd(y, pos, w, res, odt)
    ref, mag = oracle.combine(f64(y), pos.cpu().numpy(), None if w is None else f64(w), None if res is None else f64(res))
    tol = (top + 2) * U * mag + HALF[odt] * np.abs(ref) + TINY
    err = np.abs(f64(out) - ref)
    assert out.dtype == DT[odt] and (err <= tol).all(), f"{np.max(err / tol):.3g} of the tolerance"
    if rdt == odt:
        r = res.clone()
        assert m.moe_combine_fwd(y, pos, w, r, odt, out=r) is r and torch.equal(r, out)


@pytest.mark.parametrize("T,top,C", SHAPES)
@pytest.mark.parametrize("ddt,ydt,weighted", [("bf16", "bf16", True), ("f32", "f32", True), ("bf16", "f32", False),
                                              ("f32", "bf16", True)])
def test_combine_bwd(T, top, C, ddt, ydt, weighted):
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(T * C + 1)
    M = T * top + 2
    pos = places(T, top, M, T + 3 * C)
    y = torch.randn((M, C), generator=g, device="cuda").to(DT[ydt])
    dout = torch.randn((T, C), generator=g, device="cuda").to(DT[ddt])
    w = torch.randn((T, top), generator=g, device="cuda") if weighted else None
    before = torch.full((M, C), 7.0, device="cuda").to(DT[ydt])
    dy, dw = m.moe_combine_bwd(dout, pos, w, y, dy=before.clone())
    rdy, rdw, mag = oracle.combine_bwd(f64(dout), pos.cpu().numpy(), None if w is None else f64(w), f64(y), f64(before))
    tol = (HALF[ydt] + U) * np.abs(rdy) + TINY
    assert (np.abs(f64(dy) - rdy) <= tol).all()
    # a lane's share of a row's products, six additions over the wave and a few over waves
    tol = (C / 64 + 32) * U * mag + TINY
    assert (np.abs(f64(dw) - rdw) <= tol).all()
    # each gradient alone, and in place of y
    assert torch.equal(m.moe_combine_bwd(dout, pos, w, y, need_dy=False)[1], dw)
    alone, none = m.moe_combine_bwd(dout, pos, w, dy=before.clone())
    assert none is None and torch.equal(alone, dy)
    inplace = y.clone()
    got, dw2 = m.moe_combine_bwd(dout, pos, w, inplace, dy=inplace)
    here = pos[(pos >= 0) & (pos < M)].long()
    assert got is inplace and torch.equal(dw2, dw) and torch.equal(inplace[here], dy[here])
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[here] = False
    assert torch.equal(inplace[rest], y[rest])


def test_nan_stays_in_its_row():
    m = require_gpu()
    pos = torch.tensor([[0, 1], [2, -1], [3, 9]], dtype=torch.int32, device="cuda")
    y = torch.randn((4, 64), device="cuda")
    y[1, 5] = float("nan")
    y[3, 6] = float("inf")
    w = torch.ones((3, 2), device="cuda")
    w[1, 1] = w[2, 1] = float("nan")                   # of pairs without a row
    out = m.moe_combine_fwd(y, pos, w, out_dtype="f32")
    bad = ~torch.isfinite(out)
    assert bad.sum() == 2 and bad[0, 5] and bad[2, 6]
    _, dw = m.moe_combine_bwd(torch.ones((3, 64), device="cuda"), pos, w, y)
    assert torch.isfinite(dw).tolist() == [[True, False], [True, True], [False, True]]


def test_empty():
    m = require_gpu()
    pos = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    y = torch.zeros((0, 64), device="cuda")
    res = torch.randn((3, 64), device="cuda")
    assert torch.equal(m.moe_combine_fwd(y, pos, residual=res, out_dtype="f32"), res)
    assert not m.moe_combine_fwd(y, pos, out_dtype="f32").any()
    dy, dw = m.moe_combine_bwd(res, pos, None, y)
    assert dy.shape == (0, 64) and not dw.any()
    assert m.moe_dispatch(res, pos, rows=0).shape == (0, 64)
    assert m.moe_combine_fwd(y, pos[:0]).shape == (0, 64)
    assert m.moe_dispatch(res[:0], pos[:0]).shape == (0, 64)


def test_differences():
    """dy and dweights against differences of the forward kernel (linear in both, so of any step)."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.tensor([[1, 0], [3, -1]], dtype=torch.int32, device="cuda")
    y, dout, w = (torch.randn(s, generator=g, device="cuda") for s in ((4, 8), (2, 8), (2, 2)))
    dy, dw = m.moe_combine_bwd(dout, pos, w, y, dy=torch.zeros((4, 8), device="cuda"))
    loss = lambda y, w: (m.moe_combine_fwd(y, pos, w, out_dtype="f32").double() * dout.double()).sum().item()
    # 16 values below 16, rounded to 2^-20 each, over two steps of 1
    for r in range(4):
        for c in range(8):
            d = torch.zeros_like(y)
            d[r, c] = 1
            assert abs((loss(y + d, w) - loss(y - d, w)) / 2 - dy[r, c].item()) < 1e-4
    for t in range(2):
        for k in range(2):
            d = torch.zeros_like(w)
            d[t, k] = 1
            assert abs((loss(y, w + d) - loss(y, w - d)) / 2 - dw[t, k].item()) < 1e-4


def test_rows_beyond_32_bit_offsets():
    m = require_gpu()
    C, T, top = 8192, 70, 2
    M = (1 << 31) // C + 200
    pos = torch.arange(M - T * top, M, device="cuda", dtype=torch.int32).view(T, top)
    x = torch.randn((T, C), device="cuda").to(torch.bfloat16)
    xr = torch.zeros((M, C), device="cuda", dtype=torch.bfloat16)
    m.moe_dispatch(x, pos, xr=xr)
    assert torch.equal(xr[-T * top:].view(T, top, C), x[:, None].expand(-1, top, -1)) and not xr[: -T * top].any()
    w = torch.full((T, top), 0.5, device="cuda")
    assert torch.equal(m.moe_combine_fwd(xr, pos, w), x)
    dy, dw = m.moe_combine_bwd(x, pos, w, xr, dy=xr)
    assert torch.equal(xr[-T * top:].view(T, top, C), (x.float() * 0.5).to(torch.bfloat16)[:, None].expand(-1, top, -1))


def _layer(m, x, res, wn, wr, wgu, wd, G, top, valid, first=0, here=None):
    """One expert layer, forward and backward, through every entry point around its products."""
    T, C = x.shape
    here = G if here is None else here
    F = wd.shape[2]
    E = wr.shape[0]
    one = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    y, h = m.rmsnorm_fwd(x, wn, residual=res)
    logits = m.bf16_grouped_gemm_fwd(y, wr, one, E, "f32")
    ids, w, offs, row_idx, pos = m.moe_route_sort(logits, top, here, first, "sigmoid", scale=2.0, valid=valid)
    xr = m.moe_dispatch(y, pos)
    gu = m.bf16_grouped_gemm_fwd(xr, wgu, offs, 2 * F, "f32")
    gate, up = gu[:, :F], gu[:, F:]
    sg = torch.sigmoid(gate)
    act = (gate * sg * up).to(torch.bfloat16)
    yr = m.bf16_grouped_gemm_fwd(act, wd, offs, C, "bf16")
    out = m.moe_combine_fwd(yr, pos, w, h, "bf16")
    # backward of sum(out * dout)
    dout = torch.randn((T, C), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    dyr, dw = m.moe_combine_bwd(dout, pos, w, yr)
    dact = m.bf16_grouped_gemm_dgrad(dyr, wd, offs, F, "f32")
    dwd = m.bf16_grouped_gemm_wgrad(dyr, act, offs)
    dgu = torch.cat([dact * up * (sg + gate * sg * (1 - sg)), dact * gate * sg], dim=1).to(torch.bfloat16)
    dxr = m.bf16_grouped_gemm_dgrad(dgu, wgu, offs, C, "bf16")
    dwgu = m.bf16_grouped_gemm_wgrad(dgu, xr, offs)
    dlogits = m.moe_route_bwd(dw, ids, logits, "sigmoid", scale=2.0).to(torch.bfloat16)
    dy = m.moe_combine_fwd(dxr, pos, residual=m.bf16_grouped_gemm_dgrad(dlogits, wr, one, C, "f32"), out_dtype="f32")
    dx, dwn = m.rmsnorm_bwd(dy, h, wn, dres=dout)
    return {"out": out, "ids": ids, "offs": offs, "dx": dx, "dwn": dwn, "dwd": dwd, "dwgu": dwgu, "dlogits": dlogits}


def _layer_f64(x, res, wn, wr, wgu, wd, top, valid, ids, dout, first=0, here=None):
    """The same by torch's autograd in float64 on the CPU, with the experts given (the choice is not what is compared)."""
    x, res, wn, wr, wgu, wd = (t.detach().double().cpu() for t in (x, res, wn, wr, wgu, wd))
    h = (x + res).requires_grad_()
    for t in (wn, wr, wgu, wd):
        t.requires_grad_()
    y = h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + 1e-6) * wn
    p = torch.sigmoid(y @ wr.t())
    ids = ids.cpu().long()
    sel = p.gather(1, ids.clamp_min(0)) * (ids >= 0)
    w = 2.0 * sel / sel.sum(dim=1, keepdim=True).clamp_min(1e-300)
    rows = [torch.zeros_like(y[0]) for _ in range(len(y))]
    F = wd.shape[2]
    for t in range(len(y)):
        for k in range(top):
            e = int(ids[t, k]) - first
            if ids[t, k] >= 0 and 0 <= e < len(wd):
                gu = wgu[e] @ y[t]
                rows[t] = rows[t] + w[t, k] * (wd[e] @ (torch.nn.functional.silu(gu[:F]) * gu[F:]))
    out = h + torch.stack(rows)
    (out * dout.double().cpu()).sum().backward()
    return {"out": out.detach(), "dx": h.grad, "dwn": wn.grad, "dwd": wd.grad, "dwgu": wgu.grad}


@pytest.mark.parametrize("first,here", [(0, 8), (2, 3)])
def test_layer(first, here):
    """Norm, router, order, dispatch, expert products, weighted sums onto the stream, and all gradients: against
    autograd in float64; tokens of padding among them, and one GPU's experts only (the products get offs whose last is
    below the number of rows)."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(11)
    T, C, F, E, top = 50, 128, 64, 8, 3
    bf = torch.bfloat16
    x, res = (torch.randn((T, C), generator=g, device="cuda").to(bf) for _ in range(2))
    wn = 1 + 0.2 * torch.randn(C, generator=g, device="cuda")
    wr = (0.1 * torch.randn((E, C), generator=g, device="cuda")).to(bf)
    wgu = (0.1 * torch.randn((here, 2 * F, C), generator=g, device="cuda")).to(bf)
    wd = (0.1 * torch.randn((here, C, F), generator=g, device="cuda")).to(bf)
    valid = torch.ones(T, dtype=torch.bool, device="cuda")
    valid[20:24] = False
    got = _layer(m, x, res, wn, wr, wgu, wd, E, top, valid, first, here)
    dout = torch.randn((T, C), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(bf)
    hk = (x.float() + res.float()).to(bf)
    ref = _layer_f64(hk, torch.zeros_like(hk), wn, wr, wgu, wd, top, valid, got["ids"], dout, first, here)
    assert int(got["offs"][-1]) == int(((got["ids"] >= first) & (got["ids"] < first + here)).sum())
    for name, r in ref.items():
        a = got[name].detach().double().cpu()
        # a chain of at most eight bf16 roundings (2^-8 each, of independent signs over a row)
        off = (a - r).norm() / r.norm()
        assert off < 8 * 2.0 ** -8, (name, off.item())


def test_layer_in_8_bits():
    """The forward pass in 8-bit integers and in MXFP8 codes: norm with codes, dispatch of codes and scales, products."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(12)
    T, C, N, E, top = 40, 256, 128, 4, 2
    x, res = (torch.randn((T, C), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    wn = (1 + 0.2 * torch.randn(C, generator=g, device="cuda")).to(torch.bfloat16)
    w = (0.1 * torch.randn((E * N, C), generator=g, device="cuda")).to(torch.bfloat16)
    ids = torch.rand((T, E), generator=g, device="cuda").argsort(dim=1)[:, :top].int()
    offs, row_idx, pos = m.moe_sort(ids, E)
    q, s, h, y = m.int8_quantize_rmsnorm_rowwise(x, wn, residual=res, with_y=True)
    qr, sr = m.moe_dispatch(q, pos, s)
    assert torch.equal(qr, q[row_idx.long()]) and torch.equal(sr, s[row_idx.long()])
    qw, sw = m.int8_quantize_rowwise(w)
    out = m.int8_grouped_gemm_fwd(qr, sr, qw, sw, offs, N, "f32")
    group = torch.repeat_interleave(torch.arange(E), (offs[1:] - offs[:-1]).cpu().long())
    wide = (qw.double() * sw[:, None].double()).view(E, N, C).cpu()[group]
    ref = torch.bmm(wide, (qr.double() * sr[:, None].double()).cpu()[:, :, None])[:, :, 0]
    assert ((out.double().cpu() - ref).abs() <= 2.0 ** -22 * ref.abs() + 1e-30).all()

    q, s, h2, y2 = m.mx_quantize_rmsnorm_rowwise(x, wn, residual=res, with_y=True)
    assert torch.equal(h, h2) and torch.equal(y, y2)
    qr, sr = m.moe_dispatch(q, pos, s)
    mw, ms = m.mx_quantize_rowwise(w)
    out = m.mx_grouped_gemm_fwd(qr, sr, mw, ms, offs, N, "f32")
    ref, bound = oracle.mx_gemm_fwd(qr.cpu().numpy(), sr.cpu().numpy(), mw.cpu().numpy(), ms.cpu().numpy(),
                                    offs.cpu().numpy(), N)
    ok, worst, _ = oracle.check_gemm(out.cpu().numpy(), ref, bound, "f32")
    assert ok, worst


@pytest.mark.parametrize("kind", ["bf16", "int8", "mx"])
def test_products_leave_rows_behind_the_last_expert(kind):
    """offs[G] < M: rows that no expert here has stay as they were, the others are those of a call without them."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(13)
    for G, sizes, M, N, K in ((4, (3, 0, 5, 2), 40, 128, 128), (3, (300, 17, 200), 1024, 256, 384), (64, (1,) * 64, 500, 128, 256)):
        offs = torch.tensor([0, *np.cumsum(sizes)], dtype=torch.int32, device="cuda")
        n = int(offs[-1])
        x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
        dy = torch.randn((M, N), generator=g, device="cuda").to(torch.bfloat16)
        w = (0.1 * torch.randn((G * N, K), generator=g, device="cuda")).to(torch.bfloat16)
        x[n:], dy[n:] = float("nan"), float("nan")
        if kind == "bf16":
            runs = [(lambda r, o: m.bf16_grouped_gemm_fwd(x[:r], w, offs, N, "bf16", y=o), N),
                    (lambda r, o: m.bf16_grouped_gemm_dgrad(dy[:r], w, offs, K, "bf16", dx=o), K)]
            a, b = m.bf16_grouped_gemm_wgrad(dy, x, offs), m.bf16_grouped_gemm_wgrad(dy[:n], x[:n], offs)
            assert torch.isfinite(a).all() and torch.equal(a, b)
        elif kind == "int8":
            q, s = m.int8_quantize_rowwise(x)
            qw, sw = m.int8_quantize_rowwise(w)
            runs = [(lambda r, o: m.int8_grouped_gemm_fwd(q[:r], s[:r], qw, sw, offs, N, "bf16", y=o), N)]
        else:
            x[n:] = 1
            q, s = m.mx_quantize_rowwise(x)
            qw, sw = m.mx_quantize_rowwise(w)
            runs = [(lambda r, o: m.mx_grouped_gemm_fwd(q[:r], s[:r], qw, sw, offs, N, "bf16", y=o), N)]
        for call, width in runs:
            out = torch.full((M, width), 7.0, device="cuda", dtype=torch.bfloat16)
            call(M, out)
            assert (out[n:] == 7).all()
            ref = torch.empty((n, width), device="cuda", dtype=torch.bfloat16)
            call(n, ref)
            assert torch.equal(out[:n], ref)


def test_capture_and_streams():
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(14)
    T, top, C = 100, 4, 1112
    sets = []
    for s in range(2):
        pos = torch.from_numpy(np.random.default_rng(s).permutation(T * top).astype(np.int32).reshape(T, top)).cuda()
        sets.append((torch.randn((T, C), generator=g, device="cuda").to(torch.bfloat16),
                     torch.randn((T, top), generator=g, device="cuda"), pos))
    def step(x, w, pos):
        xr = m.moe_dispatch(x, pos)
        return (xr, m.moe_combine_fwd(xr, pos, w, x), *m.moe_combine_bwd(x, pos, w, xr))
    eager = [step(*s) for s in sets]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    x, w, pos = sets[0]
    xr = m.moe_dispatch(x, pos, stream=side)
    out = m.moe_combine_fwd(xr, pos, w, x, stream=side.cuda_stream)
    dy, dw = m.moe_combine_bwd(x, pos, w, xr, stream=side)
    side.synchronize()
    for a, b in zip((xr, out, dy, dw), eager[0]):
        assert torch.equal(a, b)
    graphs, outs = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(*s))
        graphs.append(graph)
    for _ in range(3):
        for graph, out, ref in zip(graphs, outs, eager):
            for o in out:
                o.zero_()
            graph.replay()
            step(*sets[1])
            torch.cuda.synchronize()
            for a, b in zip(out, ref):
                assert torch.equal(a, b)
