"""Refusals of the norm, the routing and the rows' entry points on the host (no GPU needed: validation happens before
any HIP call)."""
import pytest

from test_abi_plain import A, B, BAD, _lib, _status


def _each(L, fn, ok, bad):
    for at, value, status in bad:
        a = list(ok)
        a[at] = value
        st, msg = _status(L, fn, *a)
        assert st == status and fn in msg, (fn, at, value, st, msg)


def test_norm_refusals():
    _, L = _lib()
    #     x  xdt res rdt w wdt R  C   eps   y  ydt h  stream
    ok = [A, 1, B, 1, A, 0, 4, 64, 1e-6, A, 1, B, None]
    _each(L, "rmsnorm_fwd", ok, [(6, -1, 2), (7, 0, 2), (7, 60, 2), (7, 32776, 2), (8, 0.0, 2), (8, float("nan"), 2),
                                 (8, float("inf"), 2), (6, (1 << 40) + 1, 2), (1, 2, 4), (3, -1, 4), (5, 7, 4), (10, 2, 4),
                                 (0, None, 1), (4, None, 1), (9, None, 1), (11, None, 1), (0, BAD, 3), (2, BAD, 3),
                                 (4, BAD, 3), (9, BAD, 3), (11, BAD, 3)])
    ok[6] = 0
    assert _status(L, "rmsnorm_fwd", *ok) == (0, "")
    #     x  xdt res rdt w wdt R  C   eps   q  s  y  h  stream
    ok = [A, 1, B, 1, A, 0, 4, 64, 1e-6, A, A, A, B, None]
    for fn in ("int8_quantize_rmsnorm_rowwise", "mx_quantize_rmsnorm_rowwise"):
        _each(L, fn, ok, [(6, -1, 2), (7, 60, 2), (8, -1.0, 2), (1, 2, 4), (0, None, 1), (9, None, 1), (10, None, 1),
                          (12, None, 1), (9, BAD, 3), (10, BAD, 3), (11, BAD, 3)])
    _each(L, "mx_quantize_rmsnorm_rowwise", ok, [(7, 72, 2)])
    #     dy dydt h hdt w wdt dres R C eps dx dw ws stream
    ok = [A, 1, A, 1, A, 0, B, 4, 64, 1e-6, A, A, A, None]
    _each(L, "rmsnorm_bwd", ok, [(7, -1, 2), (8, 12, 2), (9, 0.0, 2), (1, 3, 4), (3, 3, 4), (5, 3, 4), (0, None, 1),
                                 (2, None, 1), (4, None, 1), (10, None, 1), (12, None, 1), (6, BAD, 3), (11, BAD, 3),
                                 (12, BAD, 3)])
    ok[7], ok[11] = 0, None
    assert _status(L, "rmsnorm_bwd", *ok) == (0, "")
    assert L.rmsnorm_bwd_workspace(-1, 64) == -1 and L.rmsnorm_bwd_workspace(4, 60) == -1
    assert L.rmsnorm_bwd_workspace(0, 64) == 0 and L.rmsnorm_bwd_workspace(1, 64) >= 256


def test_route_refusals():
    _, L = _lib()
    #     logits ldt bias valid T  E  top score groups keep group_top renorm scale ids w stream
    ok = [A, 0, A, None, 4, 64, 6, 0, 8, 4, 2, 1, 1.0, A, A, None]
    bad = [(4, -1, 2), (4, 1 << 30, 2), (5, 0, 2), (5, 1025, 2), (6, 0, 2), (6, 65, 2), (6, 33, 2), (8, 0, 2), (8, 5, 2),
           (9, 0, 2), (9, 9, 2), (10, 0, 2), (10, 3, 2), (12, float("inf"), 2), (12, float("nan"), 2), (1, 2, 4), (7, 2, 4),
           (7, -1, 4), (0, None, 1), (13, None, 1), (14, None, 1), (0, BAD, 3), (2, BAD, 3), (13, BAD, 3), (14, BAD, 3)]
    _each(L, "moe_route_fwd", ok, bad)
    _each(L, "moe_route_fwd", [A, 0, A, None, 4, 960, 6, 0, 80, 4, 2, 1, 1.0, A, A, None], [(7, 0, 2)])    # 80 groups
    ok[4] = 0
    assert _status(L, "moe_route_fwd", *ok) == (0, "")
    ok[4] = 4
    #                 G first offs row_idx pos ws stream
    both = ok[:-1] + [8, 8, A, A, A, A, None]
    _each(L, "moe_route_sort", both, bad + [(15, 0, 2), (15, 1025, 2), (16, -1, 2), (16, 57, 2), (17, None, 1),
                                            (18, None, 1), (19, None, 1), (18, BAD, 3)])
    #     ids T top G first offs row_idx pos ws stream
    ok = [A, 4000, 6, 8, 8, A, A, A, A, None]
    _each(L, "moe_sort", ok, [(1, -1, 2), (2, 0, 2), (2, 65, 2), (1, 1 << 29, 2), (3, 0, 2), (3, 1025, 2), (4, -1, 2),
                              (0, None, 1), (5, None, 1), (6, None, 1), (7, None, 1), (8, None, 1), (0, BAD, 3), (8, BAD, 3)])
    assert L.moe_sort_workspace(-1, 4) == -1 and L.moe_sort_workspace(4, 0) == -1 and L.moe_sort_workspace(4, 1025) == -1
    assert L.moe_sort_workspace(1 << 31, 4) == -1
    assert L.moe_sort_workspace(48, 64) == 0 and L.moe_sort_workspace(1 << 20, 64) > 0
    #     dw ids logits ldt T E top score renorm scale dlogits stream
    ok = [A, A, A, 0, 4, 64, 6, 0, 1, 1.0, B, None]
    _each(L, "moe_route_bwd", ok, [(4, -1, 2), (5, 0, 2), (5, 1025, 2), (6, 0, 2), (6, 65, 2), (9, float("nan"), 2),
                                   (3, 5, 4), (7, 5, 4), (0, None, 1), (1, None, 1), (2, None, 1), (10, None, 1),
                                   (2, BAD, 3), (10, BAD, 3)])
    ok[4] = 0
    assert _status(L, "moe_route_bwd", *ok) == (0, "")


def test_rows_refusals():
    _, L = _lib()
    #     x row_bytes scales scale_bytes pos T top M xr sr stream
    ok = [A, 64, A, 4, A, 4, 2, 8, B, B, None]
    _each(L, "moe_dispatch", ok, [(1, 0, 2), (1, 60, 2), (3, 0, 2), (3, -1, 2), (5, -1, 2), (6, 0, 2), (6, 65, 2),
                                  (5, 1 << 30, 2), (7, -1, 2), (7, 1 << 31, 2), (0, None, 1), (4, None, 1), (8, None, 1),
                                  (9, None, 1), (0, BAD, 3), (8, BAD, 3), (2, BAD, 3), (2, None, 2)])
    ok[5] = 0
    assert _status(L, "moe_dispatch", *ok) == (0, "")
    #     y ydt pos w res rdt T top M C out odt stream
    ok = [A, 1, A, A, A, 1, 4, 2, 8, 64, B, 1, None]
    _each(L, "moe_combine_fwd", ok, [(1, 2, 4), (5, 2, 4), (11, 2, 4), (6, -1, 2), (7, 0, 2), (8, -1, 2), (9, 0, 2),
                                     (9, 12, 2), (0, None, 1), (2, None, 1), (10, None, 1), (0, BAD, 3), (3, BAD, 3),
                                     (4, BAD, 3), (10, BAD, 3)])
    ok[6] = 0
    assert _status(L, "moe_combine_fwd", *ok) == (0, "")
    #     dout ddt pos w y ydt T top M C dy dw stream
    ok = [A, 1, A, A, A, 1, 4, 2, 8, 64, B, B, None]
    _each(L, "moe_combine_bwd", ok, [(1, 2, 4), (5, 2, 4), (6, -1, 2), (7, 65, 2), (8, -1, 2), (9, 12, 2), (0, None, 1),
                                     (2, None, 1), (4, None, 1), (0, BAD, 3), (3, BAD, 3), (10, BAD, 3), (11, BAD, 3)])
    ok[10] = ok[11] = None
    assert _status(L, "moe_combine_bwd", *ok) == (0, "")


def test_binding_refuses_wrong_tensors():
    m, _ = _lib()
    import torch
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    x, w = torch.zeros((4, 16), dtype=bf), torch.zeros(16)
    for call in (m.rmsnorm_fwd, m.int8_quantize_rmsnorm_rowwise, m.mx_quantize_rmsnorm_rowwise):
        with pytest.raises(ValueError, match="GPU"):
            call(x, w)
        with pytest.raises(TypeError, match="x"):
            call(x.half(), w)
        with pytest.raises(ValueError, match="w"):
            call(x, w[:8])
        with pytest.raises(ValueError, match="residual"):
            call(x, w, residual=x[:3])
        with pytest.raises(TypeError, match="h: expected"):
            call(x, w, residual=x, h=x.float())
        with pytest.raises(ValueError, match="h goes with"):
            call(x, w, h=x)
        with pytest.raises(ValueError, match="contiguous"):
            call(torch.zeros((16, 4), dtype=bf).t(), w)
    with pytest.raises(ValueError):
        m.rmsnorm_fwd(x, w, out_dtype="f16")
    with pytest.raises(TypeError, match="y"):
        m.rmsnorm_fwd(x, w, y=x.float())
    with pytest.raises(TypeError, match="dres"):
        m.rmsnorm_bwd(x, x, w, dres=x.float())
    with pytest.raises(ValueError, match="need_dw"):
        m.rmsnorm_bwd(x, x, w, dw=torch.zeros(16), need_dw=False)
    logits, ids = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=i32)
    with pytest.raises(ValueError, match="GPU"):
        m.moe_route_fwd(logits, 2)
    with pytest.raises(ValueError, match="score"):
        m.moe_route_fwd(logits, 2, "tanh")
    with pytest.raises(TypeError, match="logits"):
        m.moe_route_fwd(logits.half(), 2)
    with pytest.raises(ValueError, match="bias"):
        m.moe_route_fwd(logits, 2, bias=torch.zeros(7))
    with pytest.raises(TypeError, match="valid"):
        m.moe_route_fwd(logits, 2, valid=torch.zeros(4))
    with pytest.raises(TypeError, match="ids"):
        m.moe_sort(ids.long(), 8)
    with pytest.raises(ValueError, match="GPU"):
        m.moe_sort(ids, 8)
    with pytest.raises(ValueError, match="offs"):
        m.moe_route_sort(logits, 2, offs=torch.zeros(8, dtype=i32))
    with pytest.raises(ValueError, match="dweights"):
        m.moe_route_bwd(torch.zeros((4, 3)), ids, logits)
    with pytest.raises(TypeError, match="dlogits"):
        m.moe_route_bwd(torch.zeros((4, 2)), ids, logits, dlogits=logits.to(bf))
    with pytest.raises(ValueError, match="pos"):
        m.moe_dispatch(x, ids[:3])
    with pytest.raises(TypeError, match="x"):
        m.moe_dispatch(x.half(), ids)
    with pytest.raises(ValueError, match="scales"):
        m.moe_dispatch(x, ids, torch.zeros(3))
    with pytest.raises(ValueError, match="GPU"):
        m.moe_dispatch(x, ids, torch.zeros(4))
    with pytest.raises(ValueError, match="weights"):
        m.moe_combine_fwd(torch.zeros((8, 16)), ids, torch.zeros((4, 3)))
    with pytest.raises(ValueError, match="residual"):
        m.moe_combine_fwd(torch.zeros((8, 16)), ids, residual=torch.zeros((4, 8)))
    with pytest.raises(ValueError, match="y: expected shape"):
        m.moe_combine_bwd(x, ids, None, torch.zeros((8, 8)))
    with pytest.raises(TypeError, match="out_dtype"):
        m.moe_combine_bwd(x, ids, None, torch.zeros((8, 16)), out_dtype="bf16")
    with pytest.raises(ValueError, match="need_dy"):
        m.moe_combine_bwd(x, ids, dy=x, need_dy=False)
    with pytest.raises(TypeError, match="dy"):
        m.moe_combine_bwd(x, ids, dy=torch.zeros((8, 16), dtype=f32).half())
