"""The workspace that fp8_gemm and act_quant_gemm choose for themselves when they are captured."""
import pytest
import torch

import fp8_block_scaled_fp8bs_gb300 as fp8bs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_error():
    fp8bs.fp8bs_device_error(clear=True)
    yield
    assert fp8bs.fp8bs_device_error(clear=True) == 0


def test_captured_gemm_has_its_own_zero_filled_workspace():
    # A product that shares its last tiles over the workspace, captured twice on a stream that has seen no call. The
    # cached workspace of the stream must not be one whose zeros are only written when a graph runs.
    M, N, K = 2560, 2048, 2048
    assert fp8bs.fp8bs_gemm_plan(M, N, K, fp8bs.SCALE_FP32, True)["stream_k"]
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    b = (torch.randn(N, K, generator=g, device="cuda") * 32).to(torch.float8_e4m3fn)
    b_s = torch.rand(N // 128, K // 128, generator=g, device="cuda") / 1024
    a, a_s = fp8bs.act_quant(x)
    ref = fp8bs.fp8_gemm(a, a_s, b, b_s)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for call in (lambda: fp8bs.fp8_gemm(a, a_s, b, b_s), lambda: fp8bs.act_quant_gemm(x, b, b_s)[0]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(call())
        graphs.append(graph)
    assert (0, s.cuda_stream) not in fp8bs._workspaces
    with torch.cuda.stream(s):
        eager = fp8bs.fp8_gemm(a, a_s, b, b_s)       # before any replay
        graphs[1].replay()
        graphs[0].replay()
        graphs[1].replay()
    s.synchronize()
    assert torch.equal(eager, ref) and torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
