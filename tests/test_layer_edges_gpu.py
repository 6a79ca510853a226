"""The operators around the FP8 products of a decoder layer at the edges of what they accept."""
import pytest
import torch

import fp8_block_scaled_fp8bs_gb300 as fp8bs
from test_layer_gpu import gen, moe_weights, no_device_error, paged_case, rand  # noqa: F401

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------------- captured graphs

def attention_call(seed):
    c = paged_case(seed, [1, 1], [9000, 5000], 16, 4, 128, 128, 16)
    return lambda: fp8bs.paged_attention(**c)


def moe_call(seed):
    g = gen(seed)
    T, D, I, E = 9, 1024, 512, 16
    x, router = rand(g, T, D), rand(g, E, D, scale=0.05)
    w13, s13 = moe_weights(g, E, 2 * I, D)
    w2, s2 = moe_weights(g, E, D, I)
    return lambda: fp8bs.moe_layer(x, router, w13, s13, w2, s2, 4)


def experts_call(seed):
    g = gen(seed)
    T, D, I, E = 20, 1024, 512, 8
    x = rand(g, T, D)
    w13, s13 = moe_weights(g, E, 2 * I, D)
    w2, s2 = moe_weights(g, E, D, I)
    ids = torch.randint(0, E, (T, 2), generator=g, device="cuda", dtype=torch.int32)
    weights = torch.rand(T, 2, generator=g, device="cuda")
    return lambda: fp8bs.moe_experts(x, weights, ids, w13, s13, w2, s2)


@pytest.mark.parametrize("call", [attention_call, moe_call, experts_call])
def test_graphs_of_one_capture_stream_in_flight_at_once(call):
    # captured on the stream that all captures share, replayed side by side; and one beside eager calls on the
    # stream that it was captured on
    calls = [call(41), call(42)]
    refs = [f() for f in calls]
    capture = torch.cuda.Stream()
    graphs, outs = [], []
    for f in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=capture):
            outs.append(f())
        graphs.append(graph)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(50):
        for _ in range(4):
            for s, graph in zip(side, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for o, r in zip(outs, refs))
    for _ in range(50):
        eager = []
        for _ in range(4):
            with torch.cuda.stream(side[0]):
                graphs[0].replay()
            with torch.cuda.stream(capture):
                eager.append(calls[1]())
        torch.cuda.synchronize()
        assert torch.equal(outs[0], refs[0]) and all(torch.equal(o, refs[1]) for o in eager)


# --------------------------------------------------------------------------------------- windows

@pytest.mark.parametrize("window", [2 ** 63 - 1, 2 ** 63 - 200, 2 ** 62, 2 ** 32 + 100, 2 ** 31, 5000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("news,lens", [([1, 1], [5000, 3]), ([200, 1, 30], [300, 900, 10]), ([300], [4000])])
def test_window_longer_than_any_sequence(window, causal, news, lens):
    c = paged_case(51, news, lens, 8, 2, 128, 128, 16)
    ref = fp8bs.paged_attention(**c, causal=causal, max_kv_len=max(lens), return_lse=True)
    out = fp8bs.paged_attention(**c, causal=causal, max_kv_len=max(lens), window=window, return_lse=True)
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
