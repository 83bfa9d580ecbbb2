"""E4M3 codes of the norm where h w, or 1 / sqrt(mean h^2 + eps), leaves fp32's normal numbers: those of float64."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def codes(m, x, w, eps, what):
    q, s = m.mx_quantize_rmsnorm_rowwise(x, w, eps)
    rq, rs = oracle.rmsnorm_mx(f64(x), f64(w), eps)
    assert np.array_equal(s.cpu().numpy(), rs), f"{what}: {(s.cpu().numpy() != rs).sum()} scales differ"
    assert np.array_equal(q.cpu().numpy(), rq), f"{what}: {(q.cpu().numpy() != rq).sum()} codes differ"


@pytest.mark.parametrize("C", [256, 4096, 9216])
@pytest.mark.parametrize("xdt,wdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_products_below_normal_numbers(xdt, wdt, C):
    """h w is subnormal or vanishes and 1 / sqrt(...) lifts it back: up to 2^63 with the smallest eps."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(C)
    for eps in (2.0 ** -126, 1e-38, 1e-30, 1e-20, 2.0 ** -27, 1e-6):
        eps = max(eps, 2.0 ** -126)
        for hs, ws in ((2.0 ** -60, 2.0 ** -74), (1e-22, 1e-18), (1e-20, 1e-25), (1e-30, 1e-12), (1e-15, 1e-23), (1e-4, 1e-37),
                       (1e-3, 1e-34), (2.0 ** -62, 2.0 ** -50)):
            x = (torch.randn((6, C), generator=g, device="cuda") * hs).to(DT[xdt])
            x[4] *= torch.logspace(0, -20, C, device="cuda").to(DT[xdt])
            x[5] = 0
            x[5, ::37] = hs
            w = (torch.randn(C, generator=g, device="cuda") * ws).to(DT[wdt])
            codes(m, x, w, eps, f"eps {eps} h {hs} w {ws}")


@pytest.mark.parametrize("xdt,wdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_a_root_below_normal_numbers(xdt, wdt):
    """Rows near the types' largest values: 1 / sqrt(...) is subnormal in fp32."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(2)
    for C in (512, 8192):
        for hs in (1e37, 8e37, 1.5e38, 3e38):
            x = (torch.randn((8, C), generator=g, device="cuda").clamp(-1, 1) * hs).to(DT[xdt])
            for ws in (1e-6, 1.0, 1e6):
                w = (torch.randn(C, generator=g, device="cuda") * ws).to(DT[wdt])
                codes(m, x, w, 1e-6, f"h {hs} w {ws}")
