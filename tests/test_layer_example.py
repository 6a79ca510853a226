"""The decoder-layer example: its page bookkeeping (no GPU), and the layer run as one chunk against the same
tokens one by one."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.fixture
def example():
    return pytest.importorskip("decoder_layer")


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [dict(dim=512, q_heads=8, k_heads=2, experts=8, inter=256),
                                   dict(dim=1024, q_heads=4, k_heads=4, experts=16, inter=384, top_k=2)])
def test_layer_as_a_chunk_and_token_by_token(example, sizes):
    import torch
    layer = example.DecoderLayer(**sizes)
    n = 75
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(n + 40, sizes["dim"], generator=g, device="cuda").bfloat16()
    whole = example.Pages(32, 16)
    cache = example.new_cache(layer, 32, 16)
    # a chunk beside another sequence's
    y = layer(x, cache, whole.step({0: n, 1: 40}))
    single = example.Pages(32, 16)
    other = example.new_cache(layer, 32, 16)
    for t in range(n):
        z = layer(x[t:t + 1], other, single.step({0: 1}))
        # The same products per token, summed in another order, then rounded to bf16: the two differ where a
        # rounding (of q, k, v, o to bf16, of activations to e4m3) falls the other way, each by an ulp of its
        # format (2^-3 of a value at most for e4m3) in a few of the hundreds of terms.
        rel = (y[t].float() - z[0].float()).norm() / y[t].float().norm()
        assert float(rel) < 2e-2, (t, float(rel))
    assert torch.isfinite(y.float()).all()


def test_pages_of_a_sequence(example):
    p = example.Pages(8, 16)
    p.free, p.held, p.length = list(range(8)), {}, {}
    import torch
    real, torch.tensor = torch.tensor, lambda v, dtype=None, device=None: real(v, dtype=dtype)
    try:
        b = p.step({0: 20, 1: 3})
        assert b["kv_len"].tolist() == [20, 3] and b["q_start"].tolist() == [0, 20, 23]
        assert len(p.held[0]) == 2 and len(p.held[1]) == 1 and len(set(b["slots"].tolist())) == 23
        c = p.step({1: 1})
        assert c["positions"].tolist() == [3] and c["slots"].tolist() == [p.held[1][0] * 16 + 3]
        p.release(0)
        assert len(p.free) == 7 and 0 not in p.length
    finally:
        torch.tensor = real
