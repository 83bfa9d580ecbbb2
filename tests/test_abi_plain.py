"""Refusals of the plain-operand GEMMs, the int8 quantisers and the AdamW step on the host (no GPU needed:
validation happens before any HIP call)."""
import ctypes
import os

import pytest

A, B, BAD = 0x10000, 0x20000, 0x10001      # never dereferenced on error paths


def _lib():
    import precision_moe_expert_mx_amd as m
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmxmoe.so not built (run __graft_entry__.build())")
    return m, m.lib()


def _status(L, fn, *args):
    return getattr(L, fn)(*args), L.mxmoe_last_error().decode()


@pytest.mark.parametrize("fn", ["bf16_grouped_gemm_fwd", "bf16_grouped_gemm_dgrad", "bf16_grouped_gemm_wgrad"])
def test_bf16_gemm_refusals(fn):
    _, L = _lib()
    ok = [A, B, A, 4, 1024, 512, 256, A, 0, None]
    for at, value, status in ((3, 0, 2), (3, 1025, 2), (4, -1, 2), (4, 1 << 31, 2), (5, 0, 2), (5, 500, 2), (6, 250, 2),
                              (6, 1 << 25, 2), (8, 2, 4), (8, -1, 4), (0, None, 1), (1, None, 1), (2, None, 1),
                              (7, None, 1), (0, BAD, 3), (1, BAD, 3), (2, BAD, 3), (7, BAD, 3)):
        a = list(ok)
        a[at] = value
        st, msg = _status(L, fn, *a)
        assert st == status and fn in msg, (at, value, st, msg)
    a = list(ok)
    a[4] = 0
    if fn != "bf16_grouped_gemm_wgrad":
        assert _status(L, fn, *a) == (0, "")          # no rows: nothing to do


def test_int8_refusals():
    _, L = _lib()
    ok = [A, A, B, B, A, 4, 1024, 512, 256, A, 0, None]
    for at, value, status in ((5, 0, 2), (6, -1, 2), (7, 500, 2), (8, 264, 2), (8, 131072, 2), (10, 7, 4), (0, None, 1),
                              (1, None, 1), (2, None, 1), (3, None, 1), (4, None, 1), (9, None, 1), (0, BAD, 3),
                              (1, BAD, 3), (3, BAD, 3), (9, BAD, 3)):
        a = list(ok)
        a[at] = value
        st, msg = _status(L, "int8_grouped_gemm_fwd", *a)
        assert st == status and "int8_grouped_gemm_fwd" in msg, (at, value, st, msg)
    a = list(ok)
    a[6] = 0
    assert _status(L, "int8_grouped_gemm_fwd", *a) == (0, "")
    for fn in ("int8_quantize_rowwise", "int8_quantize_swiglu_rowwise"):
        ok = [A, 4, 64, A, A, None]
        for at, value, status in ((1, -1, 2), (2, 0, 2), (2, 60, 2), (0, None, 1), (3, None, 1), (4, None, 1), (0, BAD, 3),
                                  (3, BAD, 3), (4, BAD, 3)):
            a = list(ok)
            a[at] = value
            st, msg = _status(L, fn, *a)
            assert st == status and fn in msg, (at, value, st, msg)
        assert _status(L, fn, None, 0, 64, None, None, None) == (0, "")


def test_adamw_refusals():
    m, L = _lib()

    def call(tensors=((128, A, A, A, B, B, A, A),), gdt=0, bits=32, count=None, **hyper):
        arr = (m._AdamWTensor * max(1, len(tensors)))(*[m._AdamWTensor(*t) for t in tensors])
        h = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1, lr_dev=None, step_dev=None,
                 grad_scale=None)
        h.update(hyper)
        hyp = m._AdamWHyper(*h.values())
        return _status(L, "adamw_step", ctypes.addressof(arr), len(tensors) if count is None else count, gdt, bits,
                       ctypes.addressof(hyp), None)

    assert call(count=-1)[0] == 2 and call(bits=16)[0] == 4 and call(gdt=2)[0] == 4
    inf, nan = float("inf"), float("nan")
    for bad in (dict(lr=nan), dict(lr=inf), dict(weight_decay=nan), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=nan),
                dict(eps=0.0), dict(eps=1e-40), dict(eps=inf), dict(step=0)):
        assert call(**bad)[0] == 2, bad
    assert call(lr_dev=BAD)[0] == 3 and call(step_dev=A + 4)[0] == 3 and call(grad_scale=BAD)[0] == 3
    for at in (1, 3, 4, 5):
        t = [128, A, A, A, B, B, A, A]
        t[at] = None
        st, msg = call((t,))
        assert st == 1 and "tensor 0" in msg
        t[at] = A + 8
        assert call((t,))[0] == 3
    assert call(((128, A, A + 2, A, B, B, A, A),))[0] == 3
    assert call(((-1, A, A, A, B, B, A, A),))[0] == 2
    assert call(((128, A, A, A, B, B, None, A),), bits=8)[0] == 1
    assert call(((128, A, A, A, B, B, A, BAD),), bits=8)[0] == 3
    assert call(((0, None, None, None, None, None, None, None),)) == (0, "") and call((), count=0) == (0, "")
    assert _status(L, "adamw_step", None, 1, 0, 32, None, None)[0] == 1
    assert _status(L, "adamw_dequantize", A, A, -1, 0, A, 0, None)[0] == 2
    assert _status(L, "adamw_dequantize", A, A, 8, 2, A, 0, None)[0] == 4
    assert _status(L, "adamw_dequantize", A, A, 8, 1, A, 5, None)[0] == 4
    assert _status(L, "adamw_dequantize", A, None, 8, 1, A, 0, None)[0] == 1
    assert _status(L, "adamw_dequantize", None, None, 0, 1, None, 0, None) == (0, "")


def test_binding_refuses_wrong_tensors():
    m, _ = _lib()
    import torch
    bf, f32, i8, i32 = torch.bfloat16, torch.float32, torch.int8, torch.int32
    x, w, offs = torch.zeros((4, 16), dtype=bf), torch.zeros((2 * 8, 16), dtype=bf), torch.tensor([0, 2, 4], dtype=i32)
    with pytest.raises(ValueError, match="GPU"):
        m.bf16_grouped_gemm_fwd(x, w, offs, 8)
    with pytest.raises(TypeError):
        m.bf16_grouped_gemm_fwd(x.float(), w, offs, 8)
    with pytest.raises(TypeError):
        m.bf16_grouped_gemm_fwd(x, w, offs.long(), 8)
    with pytest.raises(ValueError, match="w: expected shape"):
        m.bf16_grouped_gemm_fwd(x, w, offs, 16)
    with pytest.raises(ValueError, match="x: expected shape"):
        m.bf16_grouped_gemm_wgrad(torch.zeros((5, 8), dtype=bf), x, offs)
    with pytest.raises(ValueError, match="output"):
        m.bf16_grouped_gemm_fwd(x, w, offs, 8, y=torch.zeros((3, 8)))
    with pytest.raises(TypeError, match="output"):
        m.bf16_grouped_gemm_fwd(x, w, offs, 8, "bf16", y=torch.zeros((4, 8)))
    with pytest.raises(ValueError):
        m.bf16_grouped_gemm_fwd(x, w, offs, 8, "f16")
    with pytest.raises(TypeError):
        m.int8_quantize_rowwise(x.float())
    with pytest.raises(ValueError):
        m.int8_quantize_swiglu_rowwise(torch.zeros((4, 15), dtype=bf))
    q, s = torch.zeros((4, 16), dtype=i8), torch.zeros(4)
    with pytest.raises(ValueError, match="sx"):
        m.int8_grouped_gemm_fwd(q, s[:3], torch.zeros((16, 16), dtype=i8), torch.zeros(16), offs, 8)
    with pytest.raises(ValueError, match="GPU"):
        m.int8_grouped_gemm_fwd(q, s, torch.zeros((16, 16), dtype=i8), torch.zeros(16), offs, 8)
    z = torch.zeros(128)
    with pytest.raises(ValueError):
        m.adamw_table([z], [z], [z], [z])               # on the CPU
    with pytest.raises(ValueError):
        m.adamw_table([], [], [], [])
    with pytest.raises(ValueError):
        m.adamw_dequantize(torch.zeros(4, dtype=torch.uint8), z[:1], "exp")
