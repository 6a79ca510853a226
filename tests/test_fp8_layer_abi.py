"""Refusals of the operators that keep a decoder layer in 8 bits: bad arguments are answered with a status before
anything touches the device (no GPU needed)."""
import ctypes

import pytest

import fp8_block_scaled_fp8bs_gb300 as fp8bs
from test_layer_abi import INVALID, MISALIGNED, OK, P, attn_args, kv, lib, norm_args  # noqa: F401


def kv8(**change):
    return kv(**{**dict(k_page_stride=4096, k_slot_stride=256, k_head_stride=128, v_page_stride=4096,
                        v_slot_stride=256, v_head_stride=128), **change})


@pytest.mark.parametrize("change,expect", [
    (dict(T=0), OK),
    (dict(T=-1), INVALID),
    (dict(T=1 << 30, cache=kv8(heads=8)), INVALID),
    (dict(v=None), INVALID),
    (dict(slots=None), INVALID),
    (dict(k=None), INVALID),
    (dict(rot_dim=24), INVALID),
    (dict(cache=kv8(page_size=8)), INVALID),
    (dict(cache=kv8(page_size=24)), INVALID),
    (dict(cache=kv8(k_slot_stride=264)), INVALID),      # 8 codes are not 16 bytes
    (dict(cache=kv8(v_head_stride=136)), INVALID),
    (dict(cache=kv8(v_page_stride=0)), INVALID),
    (dict(cache=kv8(k=None)), INVALID),
    (dict(cache=kv8(dk=120)), INVALID),
    (dict(q=P + 8), MISALIGNED),
    (dict(cache=kv8(v=P + 8)), MISALIGNED),
])
def test_qk_norm_rope_fp8_refusals(lib, change, expect):  # noqa: F811
    args = norm_args(**{**dict(cache=kv8()), **change})
    assert lib.fp8bs_qk_norm_rope_fp8(ctypes.byref(args), P, P, None) == expect


@pytest.mark.parametrize("ks,vs,expect", [(None, P, INVALID), (P, None, INVALID), (P + 2, P, MISALIGNED),
                                          (P, P + 1, MISALIGNED)])
def test_scale_pointers(lib, ks, vs, expect):  # noqa: F811
    assert lib.fp8bs_qk_norm_rope_fp8(ctypes.byref(norm_args(cache=kv8())), ks, vs, None) == expect
    assert lib.fp8bs_paged_attention_fp8(ctypes.byref(attn_args(cache=kv8())), ks, vs, None) == expect
    assert lib.fp8bs_qk_norm_rope_fp8(None, P, P, None) == INVALID
    assert lib.fp8bs_paged_attention_fp8(None, P, P, None) == INVALID


@pytest.mark.parametrize("change,expect", [
    (dict(T=0, B=0, max_q_len=0), OK),
    (dict(T=-1), INVALID),
    (dict(B=0), INVALID),
    (dict(q_heads=7), INVALID),
    (dict(window=-1), INVALID),
    (dict(max_q_len=11), INVALID),
    (dict(max_kv_len=129), INVALID),
    (dict(cache=kv8(dk=64, dv=128)), INVALID),
    (dict(cache=kv8(page_size=12)), INVALID),
    (dict(cache=kv8(k_head_stride=72)), INVALID),
    (dict(cache=kv8(pages=0)), INVALID),
    (dict(cache=kv8(v=None)), INVALID),
    (dict(q=None), INVALID),
    (dict(out=None), INVALID),
    (dict(kv_len=None), INVALID),
    (dict(page_table=None), INVALID),
    (dict(q=P + 2), MISALIGNED),
    (dict(out=P + 8), MISALIGNED),
    (dict(workspace=P + 4), MISALIGNED),
    (dict(cache=kv8(k=P + 4)), MISALIGNED),
])
def test_paged_attention_fp8_refusals(lib, change, expect):  # noqa: F811
    args = attn_args(**{**dict(cache=kv8()), **change})
    assert lib.fp8bs_paged_attention_fp8(ctypes.byref(args), P, P, None) == expect


def rms_args(**change):
    d = dict(x=P, residual=2 * P, weight=P, residual_out=3 * P, norm_out=P, y=P, s=P, x_stride=512, residual_stride=512,
             T=4, D=512, scale_fmt=0, eps=1e-6)
    d.update(change)
    return fp8bs.RmsNormArgs(**d)


@pytest.mark.parametrize("change,expect", [
    (dict(T=0), OK),
    (dict(T=-1), INVALID),
    (dict(D=0), INVALID),
    (dict(D=200), INVALID),
    (dict(D=16512), INVALID),
    (dict(x=None), INVALID),
    (dict(weight=None), INVALID),
    (dict(residual_out=None), INVALID),
    (dict(residual=None), INVALID),
    (dict(s=None), INVALID),
    (dict(y=None), INVALID),
    (dict(y=None, s=None, norm_out=None), INVALID),
    (dict(scale_fmt=2), INVALID),
    (dict(x_stride=516), INVALID),
    (dict(residual_stride=-512), INVALID),
    (dict(residual_out=P, x_stride=520), INVALID),          # in place over rows of another stride
    (dict(residual_out=2 * P, residual_stride=1024), INVALID),
    (dict(x=P + 8), MISALIGNED),
    (dict(y=P + 8), MISALIGNED),
    (dict(s=P + 2), MISALIGNED),
    (dict(norm_out=P + 2), MISALIGNED),
])
def test_rms_norm_refusals(lib, change, expect):  # noqa: F811
    assert lib.fp8bs_rms_norm(ctypes.byref(rms_args(**change)), None) == expect


def test_tensor_helpers_refuse_host_tensors():
    import torch
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fp8bs.rms_norm(x, x[0])
    codes = torch.zeros(4, 16, 4, 64).to(torch.float8_e4m3fn)
    cache = fp8bs.PagedCacheFp8(codes, codes, torch.zeros(4, 4), torch.zeros(4, 4))
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fp8bs.paged_attention(q, cache, torch.zeros(1, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                              torch.zeros(1, dtype=torch.int32))
