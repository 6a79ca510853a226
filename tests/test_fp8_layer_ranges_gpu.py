"""The operators that keep a decoder layer in 8 bits, and attention over a bf16 cache, at the ends of what they accept:
memory of any content, scores and scales of any size, slots with gaps, calls without queries. Tolerances are derived beside
each comparison."""
import pytest
import torch

import fp8_block_scaled_fp8bs_gb300 as fp8bs
from test_fp8_layer_gpu import fp8_case
from test_layer_gpu import no_device_error  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------ workspaces

def raw_args(c, out, workspace, max_q_len):
    cache, q = c["cache"], c["q"]
    k, v = cache.k, cache.v
    kv = fp8bs.KvCache(k=k.data_ptr(), v=v.data_ptr(), pages=k.shape[0], page_size=k.shape[1], heads=k.shape[2],
                       dk=k.shape[3], dv=v.shape[3], k_page_stride=k.stride(0), k_slot_stride=k.stride(1),
                       k_head_stride=k.stride(2), v_page_stride=v.stride(0), v_slot_stride=v.stride(1),
                       v_head_stride=v.stride(2))
    return fp8bs.PagedAttentionArgs(
        q=q.data_ptr(), q_token_stride=q.stride(0), q_head_stride=q.stride(1), cache=kv,
        page_table=c["page_table"].data_ptr(), table_stride=c["page_table"].stride(0), q_start=c["q_start"].data_ptr(),
        kv_len=c["kv_len"].data_ptr(), out=out.data_ptr(), lse=None, B=len(c["kv_len"]), T=q.shape[0],
        q_heads=q.shape[1], max_q_len=max_q_len, max_kv_len=c["page_table"].shape[1] * k.shape[1], window=0, causal=1,
        scale=q.shape[2] ** -0.5, workspace=None if workspace is None else workspace.data_ptr(),
        workspace_bytes=0 if workspace is None else workspace.numel())


@pytest.mark.parametrize("news,lens", [([1], [9000]), ([1] * 5, [30, 5000, 1, 700, 0]), ([1, 90, 2], [8000, 100, 40])])
@pytest.mark.parametrize("fill", [0x00, 0x01, 0x7F, 0xFF, None])
def test_a_workspace_of_any_content(news, lens, fill):
    # what a call joins is what it has written itself
    c = fp8_case(70, news, lens, 8, 2, 128, 128, 16)
    ref = fp8bs.paged_attention(**c, max_q_len=max(news))
    out = torch.empty_like(ref)
    need = fp8bs.fp8bs_paged_attention_fp8_workspace_size(raw_args(c, out, None, max(news)))
    assert need > 0
    work = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda") if fill is None else \
        torch.full((need,), fill, dtype=torch.uint8, device="cuda")
    scales = (c["cache"].k_scale.data_ptr(), c["cache"].v_scale.data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        fp8bs.fp8bs_paged_attention_fp8(raw_args(c, out, work, max(news)), *scales, stream)
        assert torch.equal(out, ref)
        out.zero_()
