"""Pins of the float64 reference of the plain-operand products, the int8 quantiser and the AdamW step
(CPU only), against brute force, library routines and hand-worked values."""
import math

import numpy as np
import pytest
import torch

import oracle
from workloads import f32_to_bf16_bits


def _bits(rng, shape):
    return f32_to_bf16_bits(rng.standard_normal(shape, dtype=np.float32))


def test_dense_products_against_sums_term_by_term():
    rng = np.random.default_rng(1)
    offs, N, K = np.array([0, 2, 2, 5], np.int32), 3, 4
    x, dy, w = _bits(rng, (5, K)), _bits(rng, (5, N)), _bits(rng, (3 * N, K))
    f = oracle.bf16_bits_to_f64
    y, ysum = oracle.dense_gemm_fwd(x, w, offs, N)
    dx, _ = oracle.dense_gemm_dgrad(dy, w, offs, N, K)
    dw, _ = oracle.dense_gemm_wgrad(dy, x, offs)
    group = [0, 0, 2, 2, 2]
    for r in range(5):
        for n in range(N):
            terms = [f(x)[r, k] * f(w)[group[r] * N + n, k] for k in range(K)]
            assert y[r, n] == pytest.approx(math.fsum(terms), rel=1e-14, abs=1e-14)
            assert ysum[r, n] == pytest.approx(math.fsum(map(abs, terms)), rel=1e-14)
        for k in range(K):
            ref = math.fsum(f(dy)[r, n] * f(w)[group[r] * N + n, k] for n in range(N))
            assert dx[r, k] == pytest.approx(ref, rel=1e-14, abs=1e-14)
    for g in range(3):
        rows = [r for r in range(5) if group[r] == g]
        for n in range(N):
            for k in range(K):
                ref = math.fsum(f(dy)[r, n] * f(x)[r, k] for r in rows)
                assert dw[g, n, k] == pytest.approx(ref, rel=1e-14, abs=1e-14)
    assert not dw[1].any()


def test_int8_rows_hand_worked():
    v = np.array([[127.0, -63.5, 0.5, 1.5, -0.5, 0.49], [0, 0, 0, 0, 0, 0], [2.0, -1.0, 1.0, 0.5, 0.0, -2.0]])
    q, s = oracle.int8_quantize_rows(v)
    assert q.tolist() == [[127, -64, 0, 2, 0, 0], [0] * 6, [127, -64, 64, 32, 0, -127]]   # ties to even
    assert s[0] == 1 and s[1] == 1 and s[2] == np.float32(2 / 127)


def test_int8_gemm_against_integers():
    rng = np.random.default_rng(2)
    offs, N, K = np.array([0, 1, 4], np.int32), 2, 16
    qx, qw = rng.integers(-128, 128, (4, K)).astype(np.int8), rng.integers(-128, 128, (2 * N, K)).astype(np.int8)
    sx, sw = rng.random(4).astype(np.float32), rng.random(2 * N).astype(np.float32)
    y = oracle.int8_gemm_fwd(qx, sx, qw, sw, offs, N)
    for r, g in enumerate([0, 1, 1, 1]):
        for n in range(N):
            acc = sum(int(a) * int(b) for a, b in zip(qx[r], qw[g * N + n]))
            assert y[r, n] == pytest.approx(acc * float(sx[r]) * float(sw[g * N + n]), rel=1e-14)


def test_second_moment_code():
    t = oracle.adamw_v_values()
    assert t[0] == 0 and t[255] == 1.875 and t[248] == 1.0 and t[1] == 1.125 * 2.0 ** -31 and t[8] == 2.0 ** -30
    assert (np.diff(t) > 0).all()
    # every value is its own code; halves between neighbours go to the even code; nothing becomes zero
    v = np.concatenate([[1.875], t[1:128]])
    q, s = oracle.adamw_pack_v(v)
    assert s[0] == 1 and q.tolist() == [255] + list(range(1, 128))
    mid = (t[1:127] + t[2:128]) / 2
    q, _ = oracle.adamw_pack_v(np.concatenate([[1.875], mid]))
    assert (q[1:] % 2 == 0).all()
    q, _ = oracle.adamw_pack_v(np.array([1.875, 1e-30, 0.0, t[1] / 3]))
    assert q.tolist() == [255, 1, 0, 1]


def test_moments_round_trip_within_half_a_step():
    rng = np.random.default_rng(3)
    for n in (1, 127, 128, 129, 1000):
        v = np.exp(rng.normal(0, 2, n))
        q, s = oracle.adamw_pack_v(v)
        assert s.shape == (-(-n // 128),)
        assert (np.abs(oracle.adamw_unpack_v(q, s) / v - 1) <= 2.0 ** -4 + 1e-6).all()
        m = rng.standard_normal(n)
        q, s = oracle.adamw_pack_m(m)
        scale = np.repeat(s.astype(np.float64), 128)[:n]
        err = np.abs(oracle.adamw_unpack_m(q, s) - m)
        assert (err <= np.maximum(np.abs(m) * 2.0 ** -4, scale * 2.0 ** -10) * (1 + 1e-6)).all()


@pytest.mark.parametrize("step", [1, 2, 50])
def test_adamw_against_torch_optimizer(step):
    """The same step as torch.optim.AdamW in float64, from the same moments."""
    rng = np.random.default_rng(4)
    p0, g, m0 = rng.standard_normal((3, 40))
    v0 = rng.random(40)
    p = torch.nn.Parameter(torch.from_numpy(p0.copy()))
    opt = torch.optim.AdamW([p], lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.3, foreach=False)
    opt.state[p] = {"step": torch.tensor(float(step - 1)), "exp_avg": torch.from_numpy(m0.copy()),
                    "exp_avg_sq": torch.from_numpy(v0.copy())}
    p.grad = torch.from_numpy(g.copy())
    opt.step()
    ref = oracle.adamw(p0, g, m0, v0, step, 0.01, 0.8, 0.95, 1e-6, 0.3)
    for got, want in zip((p.detach(), opt.state[p]["exp_avg"], opt.state[p]["exp_avg_sq"]), ref):
        np.testing.assert_allclose(got.numpy(), want, rtol=1e-12, atol=1e-14)
