"""Refusals at the ends of the plain operands' sizes, on the host (validation happens before any HIP call)."""
import ctypes

from test_abi_plain import A, B, _lib, _status


def test_adamw_tensor_longer_than_a_launch():
    m, L = _lib()
    hyper = m._AdamWHyper(1e-3, 0.9, 0.99, 1e-8, 0.0, 1, None, None, None)
    for n in ((1 << 36) - 4095, 1 << 40):
        arr = (m._AdamWTensor * 1)(m._AdamWTensor(n, A, A, A, B, B, A, A))
        st, msg = _status(L, "adamw_step", ctypes.addressof(arr), 1, 0, 32, ctypes.addressof(hyper), None)
        assert st == 2 and "2^36" in msg
