"""Refusals of the operators around the FP8 products of a decoder layer: bad arguments are answered
with a status before anything touches the device (no GPU needed), and the tensor helpers check theirs."""
import ctypes

import pytest

import fp8_block_scaled_fp8bs_gb300 as fp8bs

OK, INVALID, MISALIGNED, UNSUPPORTED, CUDA = 0, 1, 2, 3, 4
P = 0x10000            # fake, 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return fp8bs.load()


def kv(**change):
    d = dict(k=P, v=P, pages=4, page_size=16, heads=2, dk=128, dv=128, k_page_stride=4096,
             k_slot_stride=256, k_head_stride=128, v_page_stride=4096, v_slot_stride=256,
             v_head_stride=128)
    d.update(change)
    return fp8bs.KvCache(**d)


def norm_args(cache=None, **change):
    d = dict(q=P, k=P, v=P, q_token_stride=1024, q_head_stride=128, k_token_stride=256,
             k_head_stride=128, v_token_stride=256, v_head_stride=128, q_weight=P, k_weight=P, cos=P,
             sin=P, positions=P, slots=P, q_out=P, cache=cache or kv(), T=4, q_heads=8,
             max_positions=64, rot_start=0, rot_dim=128, interleaved=0, eps=1e-6)
    d.update(change)
    return fp8bs.QkNormRopeArgs(**d)


@pytest.mark.parametrize("change,expect", [
    (dict(T=-1), INVALID),
    (dict(T=0), OK),
    (dict(q=None), INVALID),
    (dict(k=None), INVALID),
    (dict(positions=None), INVALID),
    (dict(cos=None), INVALID),
    (dict(q_out=None), INVALID),
    (dict(rot_dim=24), INVALID),
    (dict(rot_dim=-16), INVALID),
    (dict(rot_start=4), INVALID),
    (dict(rot_start=16, rot_dim=128), INVALID),
    (dict(q_token_stride=1028), INVALID),
    (dict(k_head_stride=-128), INVALID),
    (dict(cache=kv(dk=120)), INVALID),
    (dict(cache=kv(dk=272)), INVALID),
    (dict(cache=kv(dv=8)), INVALID),
    (dict(cache=kv(k_slot_stride=12)), INVALID),
    (dict(cache=kv(page_size=0)), INVALID),
    (dict(cache=kv(heads=0)), INVALID),
    (dict(cache=kv(k=None)), INVALID),
    (dict(q=P + 8), MISALIGNED),
    (dict(q_out=P + 2), MISALIGNED),
    (dict(k_weight=P + 4), MISALIGNED),
    (dict(cos=P + 2), MISALIGNED),
    (dict(slots=P + 4), MISALIGNED),
    (dict(cache=kv(v=P + 8)), MISALIGNED),
])
def test_qk_norm_rope_refusals(lib, change, expect):
    assert lib.fp8bs_qk_norm_rope(ctypes.byref(norm_args(**change)), None) == expect


def attn_args(cache=None, **change):
    d = dict(q=P, q_token_stride=1024, q_head_stride=128, cache=cache or kv(), page_table=P,
             table_stride=8, q_start=P, kv_len=P, out=P, lse=P, B=2, T=10, q_heads=8, max_q_len=10,
             max_kv_len=100, window=0, causal=1, scale=0.1, workspace=P, workspace_bytes=1 << 40)
    d.update(change)
    return fp8bs.PagedAttentionArgs(**d)


@pytest.mark.parametrize("change,expect", [
    (dict(T=-1), INVALID),
    (dict(B=-1), INVALID),
    (dict(B=0), INVALID),
    (dict(T=0, B=0, max_q_len=0), OK),
    (dict(q_heads=7), INVALID),
    (dict(q_heads=0), INVALID),
    (dict(window=-1), INVALID),
    (dict(max_q_len=0), INVALID),
    (dict(max_q_len=11), INVALID),
    (dict(max_kv_len=129), INVALID),               # the table holds 8 pages of 16
    (dict(max_kv_len=1 << 31, table_stride=1 << 31), INVALID),
    (dict(cache=kv(dk=64, dv=128)), INVALID),
    (dict(cache=kv(dk=96, dv=96)), INVALID),
    (dict(cache=kv(page_size=0)), INVALID),
    (dict(cache=kv(v_head_stride=4)), INVALID),
    (dict(cache=kv(v=None)), INVALID),
    (dict(q=None), INVALID),
    (dict(out=None), INVALID),
    (dict(q_start=None), INVALID),
    (dict(page_table=None), INVALID),
    (dict(q_head_stride=100), INVALID),
    (dict(q=P + 2), MISALIGNED),
    (dict(out=P + 8), MISALIGNED),
    (dict(lse=P + 1), MISALIGNED),
    (dict(workspace=P + 4), MISALIGNED),
    (dict(cache=kv(k=P + 4)), MISALIGNED),
])
def test_paged_attention_refusals(lib, change, expect):
    assert lib.fp8bs_paged_attention(ctypes.byref(attn_args(**change)), None) == expect


def routing(**change):
    d = dict(router_w=P, bias=P, top_k=4, groups=4, topk_groups=2, score=0, normalise=1,
             route_scale=1.0)
    d.update(change)
    return fp8bs.MoeRouting(**d)


@pytest.mark.parametrize("change,size,expect", [
    ({}, dict(T=0), OK),
    ({}, dict(T=-1), INVALID),
    ({}, dict(D=100), INVALID),
    ({}, dict(D=32768), INVALID),
    ({}, dict(E=0), INVALID),
    ({}, dict(E=513), INVALID),
    (dict(top_k=0), {}, INVALID),
    (dict(top_k=33), {}, INVALID),
    (dict(groups=3), {}, INVALID),
    (dict(topk_groups=5), {}, INVALID),
    (dict(top_k=9), {}, INVALID),                  # two groups of four experts
    (dict(score=2), {}, INVALID),
    (dict(router_w=None), {}, INVALID),
    (dict(router_w=P + 2), {}, MISALIGNED),
    (dict(bias=P + 2), {}, MISALIGNED),
])
def test_moe_route_refusals(lib, change, size, expect):
    s = dict(T=3, D=256, E=16)
    s.update(size)
    assert lib.fp8bs_moe_route(P, ctypes.byref(routing(**change)), P, P, s["T"], s["D"], s["E"],
                               None) == expect
    if expect != OK or s["T"]:
        assert lib.fp8bs_moe_layer(P, ctypes.byref(routing(**change)), P, P, P, P, P, s["T"], s["D"],
                                   256, s["E"], 0, P, 1 << 40, None) == expect


@pytest.mark.parametrize("ptr,size,expect", [
    ({}, dict(T=0), OK),
    ({}, dict(T=65), INVALID),
    ({}, dict(T=-1), INVALID),
    ({}, dict(D=192), INVALID),
    ({}, dict(I=100), INVALID),
    ({}, dict(I=0), INVALID),
    ({}, dict(E=0), INVALID),
    ({}, dict(k=0), INVALID),
    ({}, dict(fmt=2), INVALID),
    ({}, dict(ws=100), INVALID),
    (dict(x=None), {}, INVALID),
    (dict(weights=None), {}, INVALID),
    (dict(ids=None), {}, INVALID),
    (dict(y=None), {}, INVALID),
    (dict(workspace=None), {}, INVALID),
    (dict(w13=P + 8), {}, MISALIGNED),
    (dict(w2=P + 1), {}, MISALIGNED),
    (dict(s2=P + 2), {}, MISALIGNED),
    (dict(ids=P + 2), {}, MISALIGNED),
])
def test_moe_experts_refusals(lib, ptr, size, expect):
    p = dict(x=P, weights=P, ids=P, w13=P, s13=P, w2=P, s2=P, y=P, workspace=P)
    p.update(ptr)
    s = dict(T=3, D=256, I=256, E=8, k=2, fmt=0, ws=1 << 40)
    s.update(size)
    assert lib.fp8bs_moe_experts(p["x"], p["weights"], p["ids"], p["w13"], p["s13"], p["w2"], p["s2"],
                                 p["y"], s["T"], s["D"], s["I"], s["E"], s["k"], s["fmt"],
                                 p["workspace"], s["ws"], None) == expect


def test_moe_workspace_size():
    small = fp8bs.fp8bs_moe_workspace_size(1, 256, 256, 8, 2)
    large = fp8bs.fp8bs_moe_workspace_size(64, 7168, 2048, 32, 8)
    assert 0 < small < large < 1 << 30
    with pytest.raises(fp8bs.Fp8bsError):
        fp8bs.fp8bs_moe_workspace_size(65, 256, 256, 8, 2)


def test_tensor_helpers_refuse_host_tensors():
    import torch
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 4, dtype=torch.int32)
    cache = fp8bs.PagedCache(torch.zeros(4, 16, 4, 64, dtype=torch.bfloat16),
                             torch.zeros(4, 16, 4, 64, dtype=torch.bfloat16))
    cos = torch.zeros(8, 32)
    with pytest.raises(TypeError):
        fp8bs.qk_norm_rope(q, q, cos, cos, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        fp8bs.paged_attention(q, cache, table, torch.zeros(2, dtype=torch.int32),
                              torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        fp8bs.moe_route(torch.zeros(2, 256, dtype=torch.bfloat16),
                        torch.zeros(8, 256, dtype=torch.bfloat16), 2)
