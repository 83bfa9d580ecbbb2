"""Pins of the float64 reference of the norm, the routing and the rows' way out and back (CPU only): hand-worked values,
torch's autograd in float64, and differences."""
import numpy as np
import pytest
import torch

import oracle


def _torch_route(x, top, score, bias, groups, keep, group_top, renorm, scale):
    """Weights as a differentiable function of logits, by torch's own softmax, sigmoid and topk."""
    p = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, dim=1)
    c = x if bias is None else p + bias
    if groups > 1:
        part = c.view(len(x), groups, -1)
        best = part.topk(min(group_top, part.shape[2]), dim=2).values.sum(dim=2)
        mask = torch.zeros_like(best).scatter(1, best.topk(keep, dim=1).indices, 1.0).bool()
        c = part.masked_fill(~mask[:, :, None], -torch.inf).view_as(x)
    ids = c.detach().topk(top, dim=1).indices
    w = p.gather(1, ids)
    return ids, scale * (w / w.sum(dim=1, keepdim=True) if renorm else w)


ROUTES = [("softmax", False, 1, 1, 1, True), ("softmax", False, 1, 1, 1, False), ("sigmoid", True, 4, 2, 2, True),
          ("sigmoid", False, 1, 1, 1, False), ("softmax", True, 2, 1, 1, False), ("softmax", False, 4, 3, 1, True)]


@pytest.mark.parametrize("score,with_bias,groups,keep,group_top,renorm", ROUTES)
def test_route_and_gradient_against_torch(score, with_bias, groups, keep, group_top, renorm):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((9, 24))
    bias = 0.2 * rng.standard_normal(24) if with_bias else None
    dw = rng.standard_normal((9, 4))
    ids, w = oracle.route(x, 4, score, bias, groups, keep, group_top, renorm, 1.5)
    tx = torch.from_numpy(x).requires_grad_()
    tids, tw = _torch_route(tx, 4, score, None if bias is None else torch.from_numpy(bias), groups, keep, group_top, renorm,
                            1.5)
    assert np.array_equal(ids, tids.numpy())
    np.testing.assert_allclose(w, tw.detach().numpy(), rtol=1e-12)
    tw.backward(torch.from_numpy(dw))
    np.testing.assert_allclose(oracle.route_bwd(dw, ids, x, score, renorm, 1.5), tx.grad.numpy(), rtol=1e-10, atol=1e-15)


def test_route_gradient_against_differences():
    rng = np.random.default_rng(2)
    x, dw = rng.standard_normal((3, 7)), rng.standard_normal((3, 2))
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, _ = oracle.route(x, 2, score, renorm=renorm)
            got = oracle.route_bwd(dw, ids, x, score, renorm)
            for t in range(3):
                for e in range(7):
                    f = []
                    for d in (1e-6, -1e-6):
                        z = x.copy()
                        z[t, e] += d
                        i2, w2 = oracle.route(z, 2, score, renorm=renorm)
                        assert np.array_equal(i2, ids)
                        f.append((w2 * dw).sum())
                    assert got[t, e] == pytest.approx((f[0] - f[1]) / 2e-6, rel=1e-6, abs=1e-9)


def test_route_ties_masks_and_padding():
    inf = np.inf
    x = np.array([[1.0, 2.0, 2.0, 2.0], [-inf, -inf, -inf, -inf], [inf, 0, inf, -inf], [0, 0, 0, 0.0]])
    ids, w = oracle.route(x, 2, valid=np.array([1, 1, 1, 0]))
    assert ids.tolist() == [[1, 2], [0, 1], [0, 2], [-1, -1]]
    assert w.tolist() == [[0.5, 0.5], [0, 0], [0.5, 0.5], [0, 0]]
    # a bias decides the choice and not the weight
    ids, w = oracle.route(np.zeros((1, 4)), 1, "sigmoid", np.array([0, 0, 0.1, 0]), renorm=False, scale=2.0)
    assert ids.tolist() == [[2]] and w.tolist() == [[1.0]]
    # the best of group 1 is the largest, but its two best together are not
    x = np.array([[3.0, 3.0, 5.0, 0.0]])
    assert oracle.route(x, 1, groups=2, keep=1, group_top=1)[0].tolist() == [[2]]
    assert oracle.route(x, 1, groups=2, keep=1, group_top=2)[0].tolist() == [[0]]


def test_sort_pairs_hand_worked():
    ids = np.array([[2, 0], [0, 3], [-1, 2]], np.int32)
    offs, row_idx, pos = oracle.sort_pairs(ids, 4)
    assert offs.tolist() == [0, 2, 2, 4, 5] and row_idx.tolist() == [0, 1, 0, 2, 1, -1]
    assert pos.tolist() == [[2, 0], [1, 4], [-1, 3]]
    offs, row_idx, pos = oracle.sort_pairs(ids, 2, first=2)
    assert offs.tolist() == [0, 2, 3] and row_idx.tolist() == [0, 2, 1, -1, -1, -1]
    assert pos.tolist() == [[0, -1], [-1, 2], [-1, 1]]


def test_norm_against_torch():
    rng = np.random.default_rng(3)
    h, w, dy, dres = rng.standard_normal((5, 16)), rng.standard_normal(16), *rng.standard_normal((2, 5, 16))
    th, tw = torch.from_numpy(h).requires_grad_(), torch.from_numpy(w).requires_grad_()
    y = torch.nn.functional.rms_norm(th, (16,), tw, 1e-3)
    np.testing.assert_allclose(oracle.rmsnorm(h, w, 1e-3)[0], y.detach().numpy(), rtol=1e-12)
    (y * torch.from_numpy(dy)).sum().backward()
    dx, dw = oracle.rmsnorm_bwd(dy, h, w, 1e-3, dres)
    np.testing.assert_allclose(dx - dres, th.grad.numpy(), rtol=1e-9, atol=1e-12)
    np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=1e-12)


def test_norm_codes():
    rng = np.random.default_rng(4)
    h, w = rng.standard_normal((6, 64)), rng.standard_normal(64)
    h[2] = 0
    y, _ = oracle.rmsnorm(h, w, 1e-6)
    q, s = oracle.rmsnorm_int8(h, w, 1e-6)
    assert (np.abs(q * s[:, None] - y) <= 0.5 * s[:, None] * (1 + 1e-12)).all() and s[2] == 1 and not q[2].any()
    q, s = oracle.rmsnorm_mx(h, w, 1e-6)
    back = oracle.mx_dequantize(q, s)
    # a block's maximum lies in [256, 512) of its scale: half a step is 2^-4 of a normal value and 2^-10 scales below
    # (2^-18 of the maximum), and a value between 448 and 512 scales becomes 448, off by less than 64 / 512 of it
    big = np.abs(y) > 448 * np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, axis=1)
    assert (np.abs(back - y) <= np.maximum(np.where(big, 2.0 ** -3, 2.0 ** -4) * np.abs(y), np.abs(y).max() * 2.0 ** -18)).all()


def test_combine_against_torch():
    rng = np.random.default_rng(5)
    T, top, C = 4, 3, 8
    pos = rng.permutation(T * top).reshape(T, top).astype(np.int32)
    pos[1, 2] = -1
    y, w, res, dout = rng.standard_normal((T * top, C)), rng.standard_normal((T, top)), *rng.standard_normal((2, T, C))
    ty, tw = torch.from_numpy(y).requires_grad_(), torch.from_numpy(w).requires_grad_()
    here = torch.from_numpy((pos >= 0).astype(np.float64))[:, :, None]
    out = torch.from_numpy(res) + (ty[torch.from_numpy(pos).long().clamp_min(0)] * tw[:, :, None] * here).sum(dim=1)
    np.testing.assert_allclose(oracle.combine(y, pos, w, res)[0], out.detach().numpy(), rtol=1e-12, atol=1e-12)
    out.backward(torch.from_numpy(dout))
    dy, dw, _ = oracle.combine_bwd(dout, pos, w, y, np.zeros_like(y))
    np.testing.assert_allclose(dy, ty.grad.numpy(), rtol=1e-12, atol=1e-15)
    np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=1e-12, atol=1e-15)


def test_softmax_weights_of_the_chosen():
    """A logit in a group that does not stay is far larger than the chosen ones, or infinite: their quotients remain."""
    for far in (60.0, 1000.0, np.inf):
        x = np.array([[far, -np.inf, 1.0, 3.0]])
        ids, w = oracle.route(x, 2, "softmax", np.array([-np.inf, -np.inf, 0, 0.5]))
        assert ids.tolist() == [[3, 2]]
        np.testing.assert_allclose(w, [[1 / (1 + np.exp(-2.0)), 1 / (1 + np.exp(2.0))]], rtol=1e-12)
        d = oracle.route_bwd(np.array([[1.0, 0.0]]), ids, x)
        np.testing.assert_allclose(d, [[0, 0, -w[0, 0] * w[0, 1], w[0, 0] * w[0, 1]]], rtol=1e-12)


def test_gradients_of_tokens_without_choices():
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            d = oracle.route_bwd(np.ones((2, 2)), np.array([[-1, -1], [7, 1]]), np.zeros((2, 4)), score, renorm)
            assert not d[0].any() and d[1].any() == (not renorm)


def test_gradients_of_vanishing_sigmoid_scores():
    """Far below 0 a sigmoid is e^x: renormalised, weights and gradients are those of a softmax over the chosen."""
    x = -500 - np.arange(5.0)[None]
    ids, w = oracle.route(x, 3, "sigmoid")
    dw = np.array([[1.0, -2.0, 0.5]])
    np.testing.assert_allclose(w, oracle.route(x, 3)[1], rtol=1e-12)
    np.testing.assert_allclose(oracle.route_bwd(dw, ids, x, "sigmoid"), oracle.route_bwd(dw, ids, x), rtol=1e-12)
