"""Offsets that end before the last row (one GPU's share of the routed rows): every product and quantiser gives what it gives
without the rows behind the last expert, and leaves the outputs' rows there as they were."""
import numpy as np
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

# experts' rows, all rows, N, K
SHARES = [((3, 0, 5, 2), 40, 256, 256), ((300, 17, 0, 200), 1024, 512, 256), ((1,) * 64, 500, 256, 512), ((0, 0, 0), 70, 256, 256)]


def data(sizes, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    offs = torch.tensor([0, *np.cumsum(sizes)], dtype=torch.int32, device="cuda")
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn((M, N), generator=g, device="cuda").to(torch.bfloat16)
    w = (0.1 * torch.randn((len(sizes) * N, K), generator=g, device="cuda")).to(torch.bfloat16)
    n = int(offs[-1])
    x[n:], dy[n:] = 1e30, -1e30
    return offs, x, dy, w, n


def rows_match(call, M, n, width, dt=torch.float32):
    """call(rows, output) with all M rows against the call with the n real ones."""
    out = torch.full((M, width), 7.0, device="cuda", dtype=dt)
    call(M, out)
    assert (out[n:] == 7).all()
    if n:
        ref = torch.empty((n, width), device="cuda", dtype=dt)
        call(n, ref)
        assert torch.equal(out[:n], ref)


def same(a, b):
    for s, t in zip(a, b):
        assert torch.equal(s, t)


@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("sizes,M,N,K", SHARES)
def test_mx(sizes, M, N, K, fast, tiled):
    m = require_gpu()
    offs, x, dy, w, n = data(sizes, M, N, K)
    G, t = len(sizes), "_tiled" if tiled else ""
    get = lambda name: getattr(m, name + t)
    cut = (lambda s, r: s[:, :r].contiguous()) if tiled else (lambda s, r: s[:r])
    (qx, sx), (qd, sd), (qw, sw) = (get("mx_quantize_rowwise")(a) for a in (x, dy, w))
    qwT, swT = get("mx_quantize_colwise")(w, None, 1, (G * N + 127) // 128 * 128)
    rows_match(lambda r, o: get("mx_grouped_gemm_fwd")(qx[:r], cut(sx, r), qw, sw, offs, N, y=o, fast=fast), M, n, N)
    rows_match(lambda r, o: get("mx_grouped_gemm_dgrad")(qd[:r], cut(sd, r), qwT, swT, offs, K, dx=o, fast=fast), M, n, K)
    ld = m.mx_colwise_ld(M, G)
    cx, cd = (get("mx_quantize_colwise")(a, offs, ld=ld) for a in (x, dy))
    if n:
        same(cx, get("mx_quantize_colwise")(x[:n], offs, ld=ld))
        dual = get("mx_quantize_dual")(x, offs, ld=ld)
        same(dual[2:], cx)
        assert torch.equal(dual[0][:n], qx[:n])
    dw = get("mx_grouped_gemm_wgrad")(*cd, *cx, offs, M, fast=fast)
    if n:
        assert torch.equal(dw, get("mx_grouped_gemm_wgrad")(*cd, *cx, offs, n, fast=fast))
    else:
        assert not dw.any()
    assert torch.isfinite(dw).all()


@pytest.mark.parametrize("sizes,M,N,K", SHARES)
def test_mx_gather_of_a_share(sizes, M, N, K):
    """row_idx as the router gives it: -1 behind the last expert."""
    m = require_gpu()
    offs, x, _, _, n = data(sizes, M, N, K)
    idx = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    idx[:n] = torch.randperm(M, device="cuda")[:n].int()
    q, s, qT, sT = m.mx_quantize_dual(x, offs, row_idx=idx)
    rows = x[idx[:n].long()]
    if n:
        same((q[:n], s[:n]), m.mx_quantize_rowwise(rows))
        same((qT, sT), m.mx_quantize_colwise(rows, offs, ld=qT.shape[1]))
    else:
        assert not qT.any() and not sT.any()


@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("sizes,M,N,K", SHARES)
def test_mx_gated_forward(sizes, M, N, K, tiled):
    """The gated forward writes what the call without those rows does, the tail of its column-wise copy included."""
    m = require_gpu()
    offs, x, dy, w, n = data(sizes, M, N, K)
    t, H = "_tiled" if tiled else "", N // 2
    get = lambda name: getattr(m, name + t)
    (qx, sx), (qw, sw) = (get("mx_quantize_rowwise")(a) for a in (x, w))
    ld = m.mx_colwise_ld(M, len(sizes))

    def outputs(r):
        u8 = lambda *shape: torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda")
        return {"y": torch.full((r, N), 7.0, device="cuda", dtype=torch.bfloat16), "qh": u8(r, H),
                "sh": u8(H // 128, r, 4) if tiled else u8(r, H // 32),
                "qhT": u8(ld // 128, H, 128) if tiled else u8(H, ld), "shT": u8(ld // 128, H, 4) if tiled else u8(H, ld // 32)}
    got = outputs(M)
    get("mx_grouped_gemm_fwd_swiglu")(qx, sx, qw, sw, offs, N, ldh=ld, **got)
    assert (got["y"][n:] == 7).all() and (got["qh"][n:] == 0x7F).all()
    if not n:                                          # (no expert has rows: nothing is written)
        assert (got["qhT"] == 0x7F).all()
        return
    ref = outputs(n)
    get("mx_grouped_gemm_fwd_swiglu")(qx[:n], sx[:, :n].contiguous() if tiled else sx[:n], qw, sw, offs, N, ldh=ld, **ref)
    for k in ("y", "qh"):
        assert torch.equal(got[k][:n], ref[k]), k
    assert torch.equal(got["sh"][:, :n] if tiled else got["sh"][:n], ref["sh"])
    for k in ("qhT", "shT"):
        assert torch.equal(got[k], ref[k]), k
    cd = get("mx_quantize_colwise")(dy, offs, ld=ld)
    dw = get("mx_grouped_gemm_wgrad")(*cd, got["qhT"], got["shT"], offs, M)
    assert torch.equal(dw, get("mx_grouped_gemm_wgrad")(*cd, ref["qhT"], ref["shT"], offs, n)) and torch.isfinite(dw).all()


@pytest.mark.parametrize("sizes,M,N,K", SHARES)
def test_mxfp4(sizes, M, N, K):
    m = require_gpu()
    offs, x, dy, w, n = data(sizes, M, N, K)
    G = len(sizes)
    (qx, sx), (qd, sd), (qw, sw) = (m.mxfp4_quantize_rowwise(a) for a in (x, dy, w))
    qwT, swT = m.mxfp4_quantize_colwise(w, None, ld=G * N)
    rows_match(lambda r, o: m.mxfp4_grouped_gemm_fwd(qx[:r], sx[:r], qw, sw, offs, N, y=o), M, n, N)
    rows_match(lambda r, o: m.mxfp4_grouped_gemm_dgrad(qd[:r], sd[:r], qwT, swT, offs, K, dx=o), M, n, K)
    ld = m.mxfp4_colwise_ld(M, G)
    cx, cd = (m.mxfp4_quantize_colwise(a, offs, ld=ld) for a in (x, dy))
    dw = m.mxfp4_grouped_gemm_wgrad(*cd, *cx, offs, M)
    if n:
        same(cx, m.mxfp4_quantize_colwise(x[:n], offs, ld=ld))
        assert torch.equal(dw, m.mxfp4_grouped_gemm_wgrad(*cd, *cx, offs, n)) and torch.isfinite(dw).all()
    else:
        assert not dw.any()


@pytest.mark.parametrize("pow2,mxk,fast", [(False, False, False), (False, False, True), (True, False, False), (True, True, False),
                                           (True, True, True)])
@pytest.mark.parametrize("sizes,M,N,K", SHARES)
def test_blockwise(sizes, M, N, K, pow2, mxk, fast):
    m = require_gpu()
    offs, x, dy, w, n = data(sizes, M, N, K)
    t = "_pow2" if mxk else ""
    get = lambda name: getattr(m, "fp8bw_grouped_gemm_" + name + t)
    qx, sx = m.fp8bw_quantize_act_1x128(x, pow2=pow2)
    qd, sd = m.fp8bw_quantize_act_1x128(dy, pow2=pow2)
    qw, sw, qwT = m.fp8bw_quantize_weight_128x128(w, transposed=True, pow2=pow2)
    rows_match(lambda r, o: get("fwd")(qx[:r], sx[:r], qw, sw, offs, N, y=o, fast=fast), M, n, N)
    rows_match(lambda r, o: get("dgrad")(qd[:r], sd[:r], qwT, sw, offs, K, dx=o, fast=fast), M, n, K)
    ld = m.fp8bw_colwise_ld_min(M, len(sizes))
    cx, cd = (m.fp8bw_quantize_colwise_128(a, offs, ld=ld, pow2=pow2) for a in (x, dy))
    dw = get("wgrad")(*cd, *cx, offs, M, fast=fast)
    if n:
        same(cx, m.fp8bw_quantize_colwise_128(x[:n], offs, ld=ld, pow2=pow2))
        assert torch.equal(dw, get("wgrad")(*cd, *cx, offs, n, fast=fast)) and torch.isfinite(dw).all()
    else:
        assert not dw.any()
