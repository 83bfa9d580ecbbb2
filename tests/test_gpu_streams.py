"""Outputs that a call on a given stream allocates are that stream's: a block that the current stream freed, and may
still be using, is not taken."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_come_from_the_stream_of_the_call(raw):
    m = require_gpu()
    G, M, N, K = 2, 4096, 512, 512
    bf16 = torch.bfloat16
    x, dy = torch.randn(M, K, device="cuda", dtype=bf16), torch.randn(M, N, device="cuda", dtype=bf16)
    w = torch.randn(G * N, K, device="cuda", dtype=bf16)
    offs = torch.tensor([0, M // 2, M], dtype=torch.int32, device="cuda")
    (q, s), (qw, sw), (mq, ms) = m.int8_quantize_rowwise(x), m.int8_quantize_rowwise(w), m.mx_quantize_rowwise(x)
    mwq, mws = m.mx_quantize_rowwise(w)
    codes, scales = torch.zeros(M * K, dtype=torch.uint8, device="cuda"), torch.zeros(M * K // 128, device="cuda")
    calls = {
        "fwd": lambda st: m.bf16_grouped_gemm_fwd(x, w, offs, N, stream=st),
        "dgrad": lambda st: m.bf16_grouped_gemm_dgrad(dy, w, offs, K, stream=st),
        "wgrad": lambda st: m.bf16_grouped_gemm_wgrad(dy, x, offs, stream=st),
        "int8": lambda st: m.int8_grouped_gemm_fwd(q, s, qw, sw, offs, N, stream=st),
        "rowwise": lambda st: m.int8_quantize_rowwise(x, stream=st)[0],
        "swiglu": lambda st: m.int8_quantize_swiglu_rowwise(x, stream=st)[0],
        "values": lambda st: m.adamw_dequantize(codes, scales, "exp_avg", stream=st),
        "mx rowwise": lambda st: m.mx_quantize_rowwise(x, stream=st)[0],
        "mx fwd": lambda st: m.mx_grouped_gemm_fwd(mq, ms, mwq, mws, offs, N, stream=st),
    }
    side = torch.cuda.Stream()
    for name, call in calls.items():
        first = call(None)
        torch.cuda.synchronize()
        kept = first.clone()
        at = first.data_ptr()
        del first                                    # the current stream's, to be used again by it alone
        out = call(side.cuda_stream if raw else side)
        side.synchronize()
        assert out.data_ptr() != at, name
        assert torch.equal(out, kept), name
        del out


def test_default_stream_given_by_its_handle():
    m = require_gpu()
    x = torch.randn(64, 512, device="cuda", dtype=torch.bfloat16)
    ref = m.int8_quantize_rowwise(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        q, s = m.int8_quantize_rowwise(x, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(q, ref[0]) and torch.equal(s, ref[1])
