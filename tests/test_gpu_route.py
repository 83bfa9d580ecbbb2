"""Routing on the GPU against its float64 reference: experts, order and rows exactly, weights and gradients within bounds
counted from the roundings of the formulas."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def spread(x):
    """Largest difference of two finite logits of a row (an exponential's relative error grows with its argument)."""
    fin = np.where(np.isfinite(x), x, np.nan)
    some = np.isfinite(fin).any(axis=1)
    d = np.zeros(len(x))
    d[some] = np.nanmax(fin[some], axis=1) - np.nanmin(fin[some], axis=1)
    return d[:, None]


def check_route(m, logits, top, score="softmax", bias=None, groups=1, keep=None, group_top=1, renorm=True, scale=1.0,
                valid=None):
    ids, w = m.moe_route_fwd(logits, top, score, bias, groups, keep, group_top, renorm, scale, valid)
    x = f64(logits)
    rid, rw = oracle.route(x, top, score, None if bias is None else f64(bias), groups, keep, group_top, renorm, scale,
                           None if valid is None else valid.cpu().numpy())
    assert np.array_equal(ids.cpu().numpy(), rid)
    # exponentials of differences (2 units, and the difference's rounding times its size), a sum of up to 1024 in at most 40
    # additions, a quotient and a product
    tol = (64 + 2 * np.minimum(spread(x), 200)) * U * np.abs(rw) + 2.0 ** -148 * abs(scale)
    err = np.abs(f64(w) - rw)
    assert (err <= tol).all(), f"weights: {np.max(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"
    return ids, w, rid, rw


CASES = [
    # T, E, top, score, bias, groups, keep, group_top, renorm, scale
    (1, 1, 1, "softmax", False, 1, None, 1, True, 1.0),
    (1, 8, 8, "sigmoid", True, 1, None, 1, True, 2.5),
    (8, 64, 6, "softmax", False, 1, None, 1, False, 1.0),
    (65, 7, 2, "softmax", True, 1, None, 1, True, 1.0),
    (130, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
    (33, 256, 8, "softmax", False, 8, 3, 1, False, 16.0),
    (100, 160, 6, "softmax", False, 8, 3, 1, False, 16.0),
    (17, 1024, 64, "sigmoid", False, 64, 5, 2, True, 1.0),
    (50, 72, 4, "sigmoid", True, 1, None, 1, False, -1.0),
    (40, 128, 10, "softmax", True, 4, 2, 2, True, 1.0),
    (29, 512, 1, "softmax", False, 1, None, 1, True, 1.0),
    (31, 384, 8, "sigmoid", True, 1, None, 1, True, 2.5),
    (9, 65, 33, "softmax", False, 1, None, 1, True, 1.0),
    (12, 60, 3, "sigmoid", True, 60, 5, 2, True, 1.0),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,top,score,with_bias,groups,keep,group_top,renorm,scale", CASES)
def test_route(T, E, top, score, with_bias, groups, keep, group_top, renorm, scale, dt):
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(T * E + top)
    for std in (1.0, 8.0):
        logits = (std * torch.randn((T, E), generator=g, device="cuda")).to(DT[dt])
        bias = 0.1 * torch.randn(E, generator=g, device="cuda") if with_bias else None
        ids, w, rid, rw = check_route(m, logits, top, score, bias, groups, keep, group_top, renorm, scale)
        dw = torch.randn((T, top), generator=g, device="cuda")
        got = m.moe_route_bwd(dw, ids, logits, score, renorm, scale)
        assert got.dtype == logits.dtype
        x, d = f64(logits), f64(dw)
        ref = oracle.route_bwd(d, rid, x, score, renorm, scale)
        # every term is a product of scores and gradients; with p the scores, w' the renormalised ones
        p = oracle.route_scores(x, score)
        q = oracle.route_scores(-x, score) if score == "sigmoid" else np.ones_like(p)      # 1 - p
        sel = np.take_along_axis(p, rid.astype(np.int64), axis=1)
        some = np.maximum(sel.sum(axis=1, keepdims=True), 1e-300) if renorm else 1.0
        wd = abs(scale) * sel / some * (np.abs(d) + ((sel / some * np.abs(d)).sum(axis=1, keepdims=True) if renorm else 0))
        size = np.zeros_like(p)
        np.put_along_axis(size, rid.astype(np.int64), wd * np.take_along_axis(q, rid.astype(np.int64), axis=1), axis=1)
        if score == "softmax" and not renorm:
            size = size + p * wd.sum(axis=1, keepdims=True)
        tol = (200 + 4 * np.minimum(spread(x), 200)) * U * size + HALF[dt] * np.abs(ref) + 2.0 ** -133
        err = np.abs(f64(got) - ref)
        assert (err <= tol).all(), f"dlogits: {np.max(err / tol):.3g} of the tolerance"


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E,groups,keep", [(64, 1, None), (256, 8, 4), (40, 1, None), (512, 4, 2)])
def test_ties_go_to_the_lower_index(score, with_bias, E, groups, keep):
    """Few distinct logits and biases: nearly every comparison is between equals."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(E)
    bias = 0.25 * torch.randint(0, 2, (E,), generator=g, device="cuda").float() if with_bias else None
    logits = torch.randint(-1, 2, (70, E), generator=g, device="cuda").float()
    logits[3] = 0
    for dt in DT.values():
        check_route(m, logits.to(dt), 8, score, bias, groups, keep, 2 if with_bias else 1)


@pytest.mark.parametrize("E,groups,keep,top", [(200, 4, 2, 8), (96, 8, 3, 10), (160, 8, 3, 6), (60, 60, 7, 5), (21, 3, 2, 4),
                                               (30, 5, 1, 6), (510, 2, 1, 9), (77, 7, 7, 3), (900, 9, 4, 12), (14, 7, 3, 6),
                                               (250, 25, 6, 16), (1000, 8, 2, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_of_any_size(E, groups, keep, top, score):
    """Groups that end inside a lane's experts, with different and with few distinct values, some of them -infinity."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(E + groups)
    T = 90
    real = torch.randn((T, E), generator=g, device="cuda")
    few = torch.randint(-2, 3, (T, E), generator=g, device="cuda").float()
    masked = real.masked_fill(torch.rand((T, E), generator=g, device="cuda") < 0.5, -torch.inf)
    bias = 0.2 * torch.randn(E, generator=g, device="cuda")
    for x in (real, few, masked):
        for dt in DT.values():
            for b in (None, bias, torch.zeros_like(bias)):
                for group_top in (1, 2):
                    check_route(m, x.to(dt), top, score, b, groups, keep, group_top, renorm=group_top == 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_nearly_equal_scores(score, with_bias):
    """Logits a few fp32 steps apart, and biases that almost make up for a difference of scores: the order is that of
    fp64."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(7)
    T, E = 200, 256
    base = torch.randint(0, 4, (T, E), generator=g, device="cuda").float()
    logits = base * (1 + torch.randint(-3, 4, (T, E), generator=g, device="cuda") * 2.0 ** -23)
    bias = None
    if with_bias:
        p = torch.sigmoid(base[0]) if score == "sigmoid" else torch.softmax(base[0], dim=0)
        bias = (p.max() - p) * (1 + torch.randint(-2, 3, (E,), generator=g, device="cuda") * 2.0 ** -23)
        logits[: T // 2] = base[0] * (1 + torch.randint(-1, 2, (T // 2, E), generator=g, device="cuda") * 2.0 ** -23)
    check_route(m, logits, 8, score, bias)
    check_route(m, logits, 8, score, bias, 8, 4, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,top,groups,keep,group_top", [(64, 6, 1, None, 1), (256, 8, 1, None, 1), (256, 8, 8, 4, 2),
                                                         (160, 6, 8, 3, 1), (1024, 12, 16, 4, 2)])
def test_scores_that_the_bias_makes_nearly_equal(score, E, top, groups, keep, group_top):
    """A bias that takes the first token's scores back to zero but for its own rounding, and tokens near that one: all
    experts, and all groups, lie within the error of fp32, far above that of fp64 (their distances are about 2^-24 p / E)."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(E + groups)
    first = torch.randn((1, E), generator=g, device="cuda")
    bias = -torch.from_numpy(oracle.route_scores(f64(first), score)[0]).float().cuda()
    near = first + torch.randn((40, E), generator=g, device="cuda") * torch.logspace(-8, -2, 40, device="cuda")[:, None]
    check_route(m, torch.cat([first, near]), top, score, bias, groups, keep, group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks_infinities_and_padding(score):
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(8)
    inf = float("inf")
    for E in (6, 64, 200):
        for dt in (torch.float32, torch.bfloat16):
            x = torch.randn((12, E), generator=g, device="cuda").to(dt)
            x[1] = -inf                                # nothing is left
            x[2, 2:] = -inf                            # fewer than top are left
            x[3] = torch.finfo(dt).min                 # the type's lowest value
            x[4, 1:] = torch.finfo(dt).min
            x[5, 5] = inf
            x[6, 2:5] = inf
            x[7] *= 1000                               # scores of 0 and 1
            x[8] = -500 - x[8].abs()                   # sigmoid scores that fp32 does not hold
            valid = torch.ones(12, dtype=torch.bool, device="cuda")
            valid[9:11] = False
            for bias in (None, torch.linspace(-0.1, 0.1, E, device="cuda")):
                for renorm in (True, False):
                    # sigmoid(-500) is 7e-218: its quotients are computed, the score itself is 0 in fp32
                    ids, w, _, rw = check_route(m, x, 4, score, bias, renorm=renorm, valid=valid)
                    assert (ids[9:11] == -1).all() and not w[9:11].any() and not w[1].any()
                    dw = torch.randn((12, 4), generator=g, device="cuda")
                    d = m.moe_route_bwd(dw, ids, x, score, renorm)
                    ok = torch.tensor([0, 2, 3, 4, 8, 9, 10, 11], device="cuda")
                    assert torch.isfinite(d).all() and not d[9:11].any() and not d[1].any()
                    assert not d[2, 2:].any()


def test_nan_gives_valid_distinct_experts():
    m = require_gpu()
    x = torch.randn((5, 64), device="cuda")
    x[1, 3] = float("nan")
    x[2] = float("nan")
    x[3, :60] = float("nan")
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(64, device="cuda")):
            for kw in ({}, {"groups": 8, "keep_groups": 2}):
                ids, w = m.moe_route_fwd(x, 6, score, bias, **kw)
                ids = ids.cpu()
                assert ((ids >= 0) & (ids < 64)).all()
                assert all(len(set(r.tolist())) == 6 for r in ids)
                if score == "sigmoid" or bias is None:           # (one NaN makes all of a row's softmax scores NaN)
                    assert 3 not in ids[1].tolist()
                assert torch.isnan(w[2]).all() and torch.isfinite(w[[0, 4]]).all()


# pairs of one block's chunk and of several, one expert, many, one GPU's, none of them here
SORTS = [(1, 1, 1, 0, 1), (8, 6, 64, 0, 64), (100, 2, 7, 0, 7), (1365, 6, 256, 0, 256), (1366, 6, 256, 96, 8),
         (5000, 8, 1024, 0, 1024), (20000, 1, 3, 1, 1), (3000, 5, 16, 12, 300), (3, 64, 64, 0, 64)]


@pytest.mark.parametrize("T,top,E,first,G", SORTS)
def test_sort(T, top, E, first, G):
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = (torch.rand((T, top), generator=g, device="cuda") ** 2 * E).int().clamp_max(E - 1)
    ids[T // 3: T // 3 + 2] = -1
    offs, row_idx, pos = m.moe_sort(ids, G, first)
    # stable sort by bucket, in numpy (the reference's loops take too long here; they are compared on small cases)
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    b = np.where((flat >= first) & (flat < first + G), flat - first, G)
    order = np.argsort(b, kind="stable")
    n = int((b < G).sum())
    want_pos = np.full(T * top, -1)
    want_pos[order[:n]] = np.arange(n)
    want_idx = np.full(T * top, -1)
    want_idx[:n] = order[:n] // top
    assert np.array_equal(offs.cpu().numpy(), np.searchsorted(np.sort(b), np.arange(G + 1)))
    assert np.array_equal(pos.cpu().numpy().reshape(-1), want_pos) and np.array_equal(row_idx.cpu().numpy(), want_idx)
    if T * top < 700:
        for got, ref in zip((offs, row_idx, pos), oracle.sort_pairs(ids.cpu().numpy(), G, first)):
            assert np.array_equal(got.cpu().numpy(), ref)


def test_sort_wild_ids():
    """ids of any value are pairs without a row, no access."""
    m = require_gpu()
    ids = torch.tensor([[2 ** 31 - 1, -2 ** 31], [5, 4], [1000000, 3]], dtype=torch.int32, device="cuda")
    for first in (0, 3, 2 ** 31 - 1):
        got = m.moe_sort(ids, 4, first)
        for a, b in zip(got, oracle.sort_pairs(ids.cpu().numpy(), 4, first)):
            assert np.array_equal(a.cpu().numpy(), b)
    d = m.moe_route_bwd(torch.ones((3, 2), device="cuda"), ids, torch.zeros((3, 6), device="cuda"), "sigmoid", False)
    assert d[0].abs().max() == 0 and d[1].tolist() == [0, 0, 0, 0, 0.25, 0.25]


def test_same_expert_twice():
    """A gradient's ids may name an expert twice: both add."""
    m = require_gpu()
    ids = torch.tensor([[1, 1, 0]], dtype=torch.int32, device="cuda")
    x, dw = torch.randn((1, 70), device="cuda"), torch.tensor([[1.0, 2.0, 3.0]], device="cuda")
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = f64(m.moe_route_bwd(dw, ids, x, score, renorm))
            ref = oracle.route_bwd(f64(dw), ids.cpu().numpy(), f64(x), score, renorm)
            assert (np.abs(got - ref) <= 2.0 ** -18 * 6).all()


@pytest.mark.parametrize("T,E,top,G,first,valid", [(8, 64, 6, 64, 0, False), (1, 8, 2, 8, 0, False), (0, 16, 2, 16, 0, False),
                                                   (2000, 256, 8, 8, 96, True), (40, 256, 8, 256, 0, True),
                                                   (3000, 60, 5, 60, 0, False), (200, 1024, 10, 100, 900, False),
                                                   (1500, 16, 6, 16, 0, True), (70, 300, 64, 300, 0, False)])
def test_route_sort_is_both(T, E, top, G, first, valid):
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(T)
    logits = torch.randn((T, E), generator=g, device="cuda")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    keep = torch.rand(T, generator=g, device="cuda") < 0.8 if valid else None
    how = dict(score="sigmoid", bias=bias, scale=2.5, valid=keep)
    if E % 8 == 0 and E // 8 * 4 >= top:
        how.update(groups=8, keep_groups=4, group_top=2)
    ids, w, *sorted_ = m.moe_route_sort(logits, top, G, first, **how)
    ids2, w2 = m.moe_route_fwd(logits, top, **how)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    for a, b in zip(sorted_, m.moe_sort(ids2, G, first)):
        assert torch.equal(a, b)
    if valid:
        assert (sorted_[2][~keep] == -1).all()


def test_streams_and_capture():
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(9)
    for T in (16, 4000):
        sets = [(torch.randn((T, 64), generator=g, device="cuda"), torch.randn((T, 6), generator=g, device="cuda"))
                for _ in range(2)]
        def step(logits, dw):
            out = m.moe_route_sort(logits, 6, renormalize=False)
            return (*out, m.moe_route_bwd(dw, out[0], logits, renormalize=False))
        eager = [step(*s) for s in sets]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        first = m.moe_route_sort(sets[0][0], 6, renormalize=False)
        at = {t.data_ptr() for t in first}
        torch.cuda.synchronize()
        del first
        got = m.moe_route_sort(sets[0][0], 6, renormalize=False, stream=side)
        side.synchronize()
        assert not at & {t.data_ptr() for t in got}    # the side stream's memory
        for a, b in zip(got, eager[0]):
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
