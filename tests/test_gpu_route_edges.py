"""Routing at the edges of its keys, masks and sizes, on the GPU against the float64 reference."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import require_gpu
from test_gpu_route import DT, HALF, U, check_route, f64, spread

pytestmark = pytest.mark.gpu


def test_a_chosen_expert_far_below_the_largest():
    """Rows whose last expert is chosen 20 and 30 below the row's largest logit, from the one group that stays."""
    m = require_gpu()
    a, b = torch.full((64,), -20.0), torch.full((64,), -1.0)
    a[56:] = torch.tensor([20.0, -10, -10, -10, -10, -10, -10, 0])
    b[56:] = torch.tensor([20.0, 0.1, 0.2, 0.3, 0.4, 0.5, 0.6, 1.0])
    x = torch.stack([a, b]).cuda()
    for score in ("softmax", "sigmoid"):
        ids = check_route(m, x, 4, score, groups=8, keep=1)[0].tolist()
        assert ids[0][:2] == [56, 63] and ids[1] == [56, 63, 62, 61]


@pytest.mark.parametrize("E,groups,keep,top", [(64, 8, 1, 4), (64, 8, 2, 5), (64, 4, 1, 6), (128, 8, 1, 8), (256, 16, 1, 3),
                                               (512, 64, 2, 6), (512, 32, 1, 16), (1024, 64, 1, 7), (1024, 64, 1, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_few_kept_experts_of_a_wide_spread(E, groups, keep, top, score):
    """At most 16 experts stay, the last group among them, and most lie far below the row's largest."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(E + groups)
    size = E // groups
    for off in (15.0, 17.0, 30.0, 50.0, 200.0):
        x = torch.randn((60, E), generator=g, device="cuda")
        x[:, E - size] += off
        x[20:40] = x[20:40].masked_fill(torch.rand((20, E), generator=g, device="cuda") < 0.4, -torch.inf)
        x[40:, E - size + 1:] -= 20.0
        for bias in (None, 0.1 * torch.randn(E, generator=g, device="cuda")):
            check_route(m, x, top, score, bias, groups, keep, 1 if bias is None else 2)


@pytest.mark.parametrize("top", [3, 17])
def test_softmax_weights_of_the_chosen(top):
    """The largest logit is in a group that does not stay: the chosen ones' quotients remain, and their gradients."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(top)
    x = torch.randn((5, 72), generator=g, device="cuda")
    x[:, 0], x[:, 1:24] = torch.tensor([0.0, 60, 1000, 1e30, float("inf")]).cuda(), -1e38
    dw = torch.randn((5, top), generator=g, device="cuda")
    for bias in (None, torch.full((72,), -0.0, device="cuda")):
        bias = bias if bias is None else bias.index_fill(0, torch.arange(24, device="cuda"), -10.0)
        for dt in (torch.float32, torch.bfloat16):
            z = x.to(dt)
            if bias is None:
                z[:, :24] = -1e38
            ids, w, rid, rw = check_route(m, z, top, "softmax", bias, 3, 1)
            assert (rid >= 24).all() and (rw > 0).all()
            d = m.moe_route_bwd(dw, ids, z).double().cpu().numpy()
            ref = oracle.route_bwd(dw.double().cpu().numpy(), rid, z.double().cpu().numpy())
            # the quotients' error as in the forward pass, the dot product's of at most 17 terms, half a step of bf16
            size = rw * (abs(dw.double().cpu().numpy()) + (rw * abs(dw.double().cpu().numpy())).sum(axis=1, keepdims=True))
            tol = 300 * 2.0 ** -24 * size.max() + (2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24) * abs(ref)
            assert (abs(d - ref) <= tol).all()


@pytest.mark.parametrize("E,groups,keep,top", [(64, 8, 3, 6), (64, 8, 3, 18), (60, 5, 2, 7), (1024, 64, 4, 12)])
def test_groups_of_both_infinities(E, groups, keep, top):
    """A group whose two best are +infinity and -infinity has no sum: it ranks last, and only `keep` groups stay."""
    m = require_gpu()
    inf = float("inf")
    size = E // groups
    g = torch.Generator(device="cuda").manual_seed(E)
    x = torch.randn((6, E), generator=g, device="cuda")
    x[:, size:2 * size] = -inf
    x[1:, size + 1] = inf                              # +inf and -inf in group 1
    x[2:, 0], x[2:, 1:size] = inf, -inf                # and in group 0
    x[4, 2 * size:] = -inf                             # (nothing else but masked ones)
    for dt in (torch.float32, torch.bfloat16):
        for score in ("softmax", "sigmoid"):
            check_route(m, x[[0, 1, 2, 3, 5]].to(dt), top, score, None, groups, keep, 2)
            ids, w, rid, rw = check_route(m, x[4:5].to(dt), top, score, None, groups, keep, 2)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    bias[:size], bias[0] = -inf, inf                   # the same by the bias
    check_route(m, torch.randn((6, E), generator=g, device="cuda"), top, "sigmoid", bias, groups, keep, 2)


@pytest.mark.parametrize("E,top,T", [(2, 1, (1 << 28) + 37), (17, 17, (1 << 26) + 5)])
def test_more_tokens_than_one_launch_holds(E, top, T):
    """16 lanes, or a wave, for each of so many tokens are more than 2^32 threads: the last tokens are those of a second
    launch, in both directions, some of them padding."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(E)
    x = torch.empty((T, E), device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    valid = torch.ones(T, dtype=torch.uint8, device="cuda")
    valid[T - 3] = valid[5] = 0
    ids = torch.full((T, top), 77, device="cuda", dtype=torch.int32)
    w = torch.full((T, top), 77.0, device="cuda")
    m.moe_route_fwd(x, top, "sigmoid", renormalize=False, valid=valid, ids=ids, weights=w)
    dl = m.moe_route_bwd(w, ids, x, "sigmoid", renormalize=False)
    step = 1 << 23
    for t in range(0, T, step):
        xs, i, ws, d = x[t:t + step], ids[t:t + step].long(), w[t:t + step], dl[t:t + step]
        real = valid[t:t + step].bool()
        assert (i[~real] == -1).all() and not ws[~real].any() and not d[~real].any()
        xs, i, ws, d = xs[real], i[real], ws[real], d[real]
        want = xs.float().sort(dim=1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(i, want)
        p = torch.sigmoid(xs.float())
        # |x| < 8: three roundings and an exponential's 2 |x| + 2 units on either side
        assert ((ws - p.gather(1, i)).abs() <= 40 * 2.0 ** -24 * ws).all()
        slope = (p * p * (1 - p)).gather(1, i)
        # (1 - p of torch's p has up to 2^-24 / (1 - p), that is e^8 units, off)
        assert ((d.float().gather(1, i) - slope).abs() <= (2.0 ** -8 + 4000 * 2.0 ** -24) * slope).all()


def check_weights(w, rw, scale=1.0):
    err = np.abs(f64(w) - rw)
    tol = 2.0 ** -19 * np.abs(rw) + 2.0 ** -149 * max(1.0, abs(scale))
    assert (err <= tol).all(), f"weights: {np.nanmax(err / tol):.3g} of the tolerance"


def check_bwd(m, x, ids, dw, score, renorm, scale=1.0):
    """moe_route_bwd against the reference: 64 units of each term (scores as the weights, 32; their differences, products and
    sums over at most 16 choices), for the softmax that is not renormalised 2 |x - max| more, and half a step of bf16."""
    got, z, d, rid = f64(m.moe_route_bwd(dw, ids, x, score, renorm, scale)), f64(x), f64(dw), ids.cpu().numpy()
    ref = oracle.route_bwd(d, rid, z, score, renorm, scale)
    p = oracle.route_scores(z, score)
    q = oracle.route_scores(-z, score) if score == "sigmoid" else np.ones_like(p)
    here = rid >= 0
    at = np.where(here, rid, 0).astype(np.int64)
    sel = oracle.route_scores(np.take_along_axis(z, at, axis=1), score) if renorm and score == "softmax" else np.take_along_axis(p, at, axis=1)
    sel = np.where(here, sel, 0.0)
    w = sel / np.maximum(sel.sum(axis=1, keepdims=True), 1e-300) if renorm else sel
    term = abs(scale) * w * (np.abs(d) + ((w * np.abs(d)).sum(axis=1, keepdims=True) if renorm else 0))
    size = np.zeros_like(p)
    np.add.at(size, (np.arange(len(z))[:, None], at), np.where(here, term * np.take_along_axis(q, at, axis=1), 0.0))
    units = np.full((len(z), 1), 64.0)
    if score == "softmax" and not renorm:
        size = size + p * term.sum(axis=1, keepdims=True)
        units = units + 2 * np.minimum(spread(z), 200)
    tol = units * U * size + HALF["bf16" if x.dtype == torch.bfloat16 else "f32"] * np.abs(ref) + 2.0 ** -133
    if score == "softmax" and not renorm:              # (a score below 2^-126 of an expert that was not chosen counts as 0)
        tol = tol + 2.0 ** -126 * term.sum(axis=1, keepdims=True)
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"dlogits, {score} {renorm} {scale} {x.dtype}: {np.max(err / tol):.3g} of the tolerance"


@pytest.mark.parametrize("E,top", [(64, 6), (256, 8), (512, 16), (1000, 16), (40, 33)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_small_weights_are_as_exact_as_large_ones(E, top, score):
    """Chosen logits up to 100 below the largest, down to weights that are subnormal in fp32."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(E)
    T = 120
    x = torch.randn((T, E), generator=g, device="cuda") - torch.linspace(0, 90, T, device="cuda")[:, None]
    x[:, 3] += torch.linspace(0, 90, T, device="cuda") if score == "softmax" else 0
    bias = torch.zeros(E, device="cuda")
    bias[3] = 1.0                                      # (always chosen)
    for dt in DT.values():
        for b in (None, bias):
            for renorm in (True, False):
                for scale in (1.0, 2.5):
                    z = x.to(dt)
                    ids, w = m.moe_route_fwd(z, top, score, b, renormalize=renorm, scale=scale)
                    rid, rw = oracle.route(f64(z), top, score, None if b is None else f64(b), renorm=renorm, scale=scale)
                    assert np.array_equal(ids.cpu().numpy(), rid)
                    check_weights(w, rw, scale)
                    check_bwd(m, z, ids, torch.randn((T, top), generator=g, device="cuda"), score, renorm, scale)


@pytest.mark.parametrize("E,groups,keep,top", [(64, 1, None, 6), (256, 8, 4, 8), (1000, 1, None, 12), (60, 1, None, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_that_switch_experts_off(E, groups, keep, top, score):
    """A bias of -infinity, of the type's lowest value or of 1e30 and more keeps experts out, or in, of every token."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(E)
    x = torch.randn((50, E), generator=g, device="cuda")
    for off in (float("-inf"), torch.finfo(torch.float32).min, -1e30, -1e4):
        bias = 0.1 * torch.randn(E, generator=g, device="cuda")
        bias[torch.rand(E, generator=g, device="cuda") < 0.3] = off
        for dt in DT.values():
            ids, w, _, rw = check_route(m, x.to(dt), top, score, bias, groups, keep, 2 if groups > 1 else 1)
            assert (bias[ids.long()] > -1).all()
            check_weights(w, rw)
    bias[5], bias[9] = float("inf"), 1e30
    ids = check_route(m, x, top, score, bias)[0]
    assert (ids[:, 0] == 5).all() and (ids[:, 1] == 9).all()


@pytest.mark.parametrize("E,groups,keep,top", [(64, 1, None, 6), (256, 8, 4, 8), (256, 8, 2, 16), (72, 9, 3, 8), (16, 2, 1, 8),
                                               (60, 1, None, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_fewer_experts_than_are_chosen(E, groups, keep, top, score):
    """Most or all experts are kept out by -infinity, some logits are equal or masked: the index decides among those out."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(E)
    for part in (0.5, 0.95, 1.0):
        x = torch.randn((30, E), generator=g, device="cuda")
        x[10:] = torch.randint(-2, 3, (20, E), generator=g, device="cuda").float()
        x[20:, ::3] = -torch.inf
        bias = 0.1 * torch.randn(E, generator=g, device="cuda")
        bias[torch.rand(E, generator=g, device="cuda") < part] = -torch.inf
        for dt in DT.values():
            for group_top in (1, 2):
                check_route(m, x.to(dt), top, score, bias, groups, keep, group_top)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_two_best_of_a_group(dt):
    """group_top=2 sums logits without a bias, and scores with one: here they prefer different groups."""
    m = require_gpu()
    x = torch.tensor([[10.0, 0.125, 4.0, 4.0]], device="cuda").to(DT[dt])
    for score, first in (("sigmoid", [2, 3]), ("softmax", [0, 1])):
        assert check_route(m, x, 2, score, None, 2, 1, 2)[0].tolist() == [[0, 1]]
        assert check_route(m, x, 2, score, torch.zeros(4, device="cuda"), 2, 1, 2)[0].tolist() == [first]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradients_of_masked_rows(score):
    """Values of the gradients where logits are masked, infinite or far apart, and of tokens of padding."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(8)
    inf = float("inf")
    for E in (6, 64, 200):
        for dt in (torch.float32, torch.bfloat16):
            x = torch.randn((12, E), generator=g, device="cuda").to(dt)
            x[1] = -inf
            x[2, 2:] = -inf
            x[3] = torch.finfo(dt).min
            x[4, 1:] = torch.finfo(dt).min
            x[5, 5] = inf
            x[6, 2:5] = inf
            x[7] *= 1000
            x[8] = -500 - x[8].abs()
            valid = torch.ones(12, dtype=torch.bool, device="cuda")
            valid[9:11] = False
            for bias in (None, torch.linspace(-0.1, 0.1, E, device="cuda")):
                for renorm in (True, False):
                    ids, w, _, rw = check_route(m, x, 4, score, bias, renorm=renorm, valid=valid)
                    check_weights(w, rw)
                    check_bwd(m, x, ids, torch.randn((12, 4), generator=g, device="cuda"), score, renorm)


def test_as_many_pairs_as_there_may_be():
    """2^31 - 1 tokens, one choice each: token, pair and row numbers up to the largest int32."""
    m = require_gpu()
    T, step = 2 ** 31 - 1, 1 << 26
    x = torch.empty((T, 2), device="cuda", dtype=torch.bfloat16)
    for t in range(0, T, step):
        x[t:t + step].normal_(generator=torch.Generator(device="cuda").manual_seed(t))
    ids, w, offs, row_idx, pos = m.moe_route_sort(x, 1, score="sigmoid", renormalize=False)
    del w
    done = [0, 0]
    n0 = int(offs[1])
    assert offs.tolist() == [0, n0, T]
    for t in range(0, T, step):
        i = (x[t:t + step, 1] > x[t:t + step, 0]).long()
        assert torch.equal(ids[t:t + step, 0].long(), i)
        here = torch.arange(t, min(T, t + step), device="cuda")
        for e in (0, 1):
            mine = here[i == e]
            first = e * n0 + done[e]
            want = torch.arange(first, first + len(mine), device="cuda")
            assert torch.equal(pos[t:t + step, 0][i == e].long(), want)
            assert torch.equal(row_idx[first:first + len(mine)].long(), mine)
            done[e] += len(mine)
    assert done == [n0, T - n0]
