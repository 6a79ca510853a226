"""The operators that keep a decoder layer in 8 bits, and attention over a bf16 cache, at the ends of what they accept:
memory of any content, scores and scales of any size, slots with gaps, calls without queries. Tolerances are derived beside
each comparison."""
import math
import random

import pytest
import torch

import fp8_block_scaled_fp8bs_gb300 as fp8bs
from test_fp8_layer_gpu import SHAPES, copy, empty_cache, fp8_case, fp8_check, power_above, same, write_inputs
from test_layer_gpu import attention_check, gen, no_device_error, norm_rope_ref, paged_case, rand  # noqa: F401

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
LOG2E = 1 / math.log(2)


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


# ------------------------------------------------------------------------------------ sizes of scores

def level_case(codes, news, lens, hq, hk, dk, dv, low, high):
    """Keys that are all alike, so that each row's scores are one number, of low .. high in units of log2 and either
    sign from row to row: o is the mean of the values, however coarse binary32 is there."""
    case = fp8_case(71, news, lens, hq, hk, dk, dv, 16, poison=False, k_spread=0, v_spread=0) if codes else \
        paged_case(71, news, lens, hq, hk, dk, dv, 16, poison=False)
    g = gen(72)
    k = case["cache"].k
    row = (torch.rand(hk, dk, generator=g, device="cuda") * 100 + 20).to(E4M3)
    if codes:
        k.view(torch.uint8)[:] = row.view(torch.uint8)
        case["cache"].k_scale.fill_(1.0)
    else:
        k[:] = row.bfloat16()
    q = torch.rand(case["q"].shape, generator=g, device="cuda", dtype=torch.float64) + 0.5
    size = torch.rand(q.shape[:2], generator=g, device="cuda", dtype=torch.float64)
    size = torch.exp2(low + (high - low) * size)
    size[:, ::2] *= -1
    s = (q * row.double().repeat_interleave(hq // hk, 0)).sum(-1) * (dk ** -0.5 * LOG2E)
    case["q"] = (q * (size / s)[..., None]).bfloat16()
    return case, row


def check_level(codes, news, lens, hq, hk, dk, dv, low, high, window=0):
    c, row = level_case(codes, news, lens, hq, hk, dk, dv, low, high)
    out, lse = fp8bs.paged_attention(**c, max_q_len=max(news), window=window, return_lse=True)
    cache, t = c["cache"], 0
    for b, (n, L) in enumerate(zip(news, lens)):
        j = torch.arange(L, device="cuda")
        pg = c["page_table"][b].long()[j // 16]
        if codes:
            v = cache.v.view(torch.uint8)[pg, j % 16].view(E4M3).double() * cache.v_scale.double()[pg][..., None]
        else:
            v = cache.v[pg, j % 16].double()
        v = v.repeat_interleave(hq // hk, 1)
        q = c["q"][t:t + n].double()
        terms = q * row.double().repeat_interleave(hq // hk, 0)
        s = terms.sum(-1) * dk ** -0.5
        last = L - n + 1 + torch.arange(n, device="cuda")
        first = (last - window).clamp(min=0) if window else torch.zeros_like(last)
        count = last - first

        def mean(x):
            sums = torch.cat([torch.zeros_like(x[:1]), x.cumsum(0)])
            return (sums[last] - sums[first]) / count[:, None, None]

        o, mag = mean(v), mean(v.abs())
        # the probabilities of a row are all the same number: one rounding of it to bf16, or to two e4m3 numbers (2^-8)
        # and one of the output (2^-8); binary32 sums 2^-12
        err = (out[t:t + n].double() - o).abs()
        assert bool((err <= (2.0 ** -7 + 2.0 ** -12) * mag).all()), float((err / mag).nan_to_num(math.inf).max())
        # a score: queries to 2^-17 of their largest channel, binary32 sums of 192 terms 2^-16 of them; then three
        # roundings of the sum, 2^-20
        size = (c["q"][t:t + n].double().abs().amax(-1) * row.double().sum(-1).repeat_interleave(hq // hk)) * dk ** -0.5
        l = s + count.double().log()[:, None]
        far = size * (2.0 ** -17 + 2.0 ** -16) + 2.0 ** -20 * l.abs() + 1e-5
        assert bool(((lse[t:t + n].double() - l).abs() <= far).all())
        t += n


LEVELS = [([1, 1, 1, 1, 2], [1, 2, 40, 300, 129]), ([1], [20000]), ([130, 1, 3], [600, 1, 5]), ([300], [400]),
          ([40], [9000])]


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("news,lens", LEVELS)
@pytest.mark.parametrize("low,high", [(20, 26), (26, 29), (29, 40)])
def test_scores_of_any_size_over_codes(dk, dv, news, lens, low, high):
    check_level(True, news, lens, 16, 2, dk, dv, low, high)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("window", [1, 70, 200])
def test_scores_of_any_size_in_windows(codes, dk, dv, window):
    # far rows beside others, tiles that are masked at both ends
    for news, lens in LEVELS:
        check_level(codes, news, lens, 16, 2, dk, dv, 18, 36, window)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("low,high", [(10, 24), (24, 40)])
def test_one_key_far_above_the_others(codes, dk, dv, low, high):
    # one key of each sequence, in its middle, is twice the others: it is all that a row of positive scores has, and
    # nothing to a row of negative ones, before which and after which its scores are alike
    for news, lens in (([1, 1, 3], [300, 2, 900]), ([1], [9000]), ([200, 1], [700, 40]), ([300], [1000])):
        c, row = level_case(codes, news, lens, 16, 2, dk, dv, low, high)
        cache, t = c["cache"], 0
        keys = cache.k.view(torch.uint8) if codes else cache.k
        twice = (row.float() * 2).to(E4M3).view(torch.uint8) if codes else (row.float() * 2).bfloat16()
        for b, L in enumerate(lens):
            keys[int(c["page_table"][b, L // 2 // 16]), L // 2 % 16] = twice
        out, lse = fp8bs.paged_attention(**c, max_q_len=max(news), return_lse=True)
        for b, (n, L) in enumerate(zip(news, lens)):
            j = torch.arange(L, device="cuda")
            pg = c["page_table"][b].long()[j // 16]
            if codes:
                v = cache.v.view(torch.uint8)[pg, j % 16].view(E4M3).double() * cache.v_scale.double()[pg][..., None]
            else:
                v = cache.v[pg, j % 16].double()
            v = v.repeat_interleave(8, 1)
            star = (j == L // 2).double()
            seen = (j <= L - n + torch.arange(n, device="cuda")[:, None]).double()
            low_w, high_w = seen * (1 - star), seen * star
            has = high_w.sum(1, keepdim=True)
            w = torch.where(has > 0, high_w, low_w / low_w.sum(1, keepdim=True).clamp(min=1))       # positive rows
            u = torch.where(low_w.sum(1, keepdim=True) > 0, low_w / low_w.sum(1, keepdim=True).clamp(min=1), high_w)
            positive = (torch.arange(16, device="cuda") % 2 == 1)[:, None, None]
            p = torch.where(positive, w, u)                                                          # [heads, n, keys]
            o, mag = (torch.einsum("hnk,khd->nhd", p, x) for x in (v, v.abs()))
            # scores are 2^10 and more apart, so that nothing is left to the other keys; one rounding of the probabilities,
            # one of the output, binary32 sums
            err = (out[t:t + n].double() - o).abs()
            assert bool((err <= (2.0 ** -7 + 2.0 ** -12) * mag).all()), float((err / mag).nan_to_num(math.inf).max())
            t += n


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("news,lens", LEVELS)
def test_scores_at_the_ends_of_binary32(dk, dv, news, lens):
    check_level(True, news, lens, 16, 2, dk, dv, 127.84, 127.95)


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("news,lens", LEVELS)
@pytest.mark.parametrize("low,high", [(20, 29), (29, 40)])
def test_scores_of_any_size_over_bf16(dk, dv, news, lens, low, high):
    check_level(False, news, lens, 16, 2, dk, dv, low, high)


# ------------------------------------------------------------------------- sizes of queries, keys, scale

@pytest.mark.parametrize("size,unit", [(1e-28, 2.0 ** 85), (2.0 ** -115, 2.0 ** 110), (1e25, 2.0 ** -90)])
def test_small_queries_over_large_keys(size, unit):
    for news, lens in (([1, 3], [500, 200]), ([1, 130], [500, 200])):
        c = fp8_case(73, news, lens, 8, 2, 128, 128, 16, k_spread=0)
        c["cache"].k_scale.fill_(unit)
        c["q"] = (c["q"].double() * (size * 2.0 ** -7)).bfloat16()
        fp8_check(c, news, lens, scale=128 ** -0.5 / (size * unit))
        fp8_check(c, news, lens, scale=0.0)


def test_scale_of_zero_over_large_queries():
    for news, lens in (([1, 3], [500, 200]), ([1, 130], [500, 200])):
        c = fp8_case(74, news, lens, 8, 2, 128, 128, 16, k_spread=0)
        c["q"] = (c["q"].double() * 1e25).bfloat16()
        fp8_check(c, news, lens, scale=0.0)


def test_scale_of_zero_over_large_bf16_keys():
    for news, lens in (([1, 3], [500, 200]), ([1, 130], [500, 200]), ([300], [400])):
        c = paged_case(75, news, lens, 8, 2, 128, 128, 16)
        c["q"] = (c["q"].double() * 1e18).bfloat16()
        c["cache"].k.copy_((c["cache"].k.double() * 1e18).bfloat16())
        attention_check(c, news, lens, scale=0.0)


@pytest.mark.parametrize("mean,size", [(-33, 1.0), (20, 2.0 ** -8), (73, 2.0 ** -8)])
def test_value_scales_at_the_ends_of_their_range(mean, size):
    # scales within 2^80 of one another, from 2^-80 and up to 2^113
    for news, lens in (([1, 3], [500, 200]), ([1, 130], [500, 200]), ([1], [9000])):
        c = fp8_case(78, news, lens, 8, 2, 128, 128, 16, poison=False, k_spread=0, v_spread=40)
        c["cache"].v_scale.mul_(2.0 ** mean)
        c["cache"].v.copy_((c["cache"].v.float() * size).to(E4M3))
        fp8_check(c, news, lens, scale=0.01)


# ------------------------------------------------------------------------------ writes without queries

def test_write_without_queries_reports_bad_indices():
    page, hk, d = 16, 3, 64
    for T, bad in ((5, 1), (200, 199), (200, 0), (600, 300)):
        for pos, slot, want in ((4000, None, fp8bs.DEVERR_INDEX), (-1, None, fp8bs.DEVERR_INDEX),
                                (None, 41 * page, fp8bs.DEVERR_INDEX), (None, -1, 0)):
            cache = empty_cache(41, page, hk, d, d)
            x = write_inputs(76, T, 0, hk, d, d, 32, True)
            slots = torch.arange(page, page + T, device="cuda")
            if pos is not None:
                x["pos"][bad] = pos
            if slot is not None:
                slots[bad] = slot
            q = fp8bs.qk_norm_rope(x["q"], x["k"], x["cos"], x["sin"], x["pos"], q_weight=x["qw"], k_weight=x["kw"],
                                   cache=cache, v=x["v"], slots=slots)
            assert q.shape == (T, 0, d)
            assert fp8bs.fp8bs_device_error(clear=True) == want


# ------------------------------------------------------------------------------------ rows of one token

def test_norm_of_one_row_in_place_whatever_its_stride():
    g = gen(77)
    D = 640
    wide, w = rand(g, 4, D + 264), rand(g, D)
    for i in range(2):
        x, r = wide[:1, 8:8 + D], rand(g, 3, 2 * D)[:1, :D]
        ref = fp8bs.rms_norm(x.clone(), w, residual=r.clone(), quant="fp32", norm=True)
        out = (x, r)[i]
        got = fp8bs.rms_norm(x, w, residual=r, quant="fp32", norm=True, residual_out=out)
        assert got.h.data_ptr() == out.data_ptr() and all(same(a, b) for a, b in zip(got, ref))


# ------------------------------------------------------------------------------------- slots with gaps

def gaps_check(cache, x, runs):
    """A write of one run a page, runs[page] = its rising slots of the page, against the definition."""
    page, hk = cache.k.shape[1:3]
    before = copy(cache)
    slots = torch.tensor([pg * page + o for pg, at in runs.items() for o in at], device="cuda")
    fp8bs.qk_norm_rope(x["q"], x["k"], x["cos"], x["sin"], x["pos"], q_weight=x["qw"], k_weight=x["kw"], cache=cache,
                       v=x["v"], slots=slots)
    rk = norm_rope_ref(x["k"], x["kw"], x["cos"], x["sin"], x["pos"], 0, False, 1e-6)
    t = 0
    for pg, at in runs.items():
        rows = torch.arange(t, t + len(at), device="cuda")
        t += len(at)
        for name, want, exact in (("k", rk[rows], False), ("v", x["v"][rows].double(), True)):
            codes, scale = getattr(cache, name)[pg], getattr(cache, name + "_scale")[pg].double()
            old, kept = getattr(before, name)[pg], getattr(before, name + "_scale")[pg].double()
            if at[0] == 0:
                kept = torch.zeros_like(kept)
            # (binary32: where the largest is within 2^-17 of a border, the power of two beside it)
            need = want.abs().amax((0, 2)).clamp(min=1e-4) / 448
            low = torch.maximum(kept, power_above(need * (1 - 2.0 ** -17)))
            assert bool(((scale == low) | (scale == torch.maximum(kept, power_above(need * (1 + 2.0 ** -17))))).all())
            if exact:
                assert same(codes[at], (want / scale[:, None]).float().to(E4M3))
            else:
                # half a step, and the binary32 terms of norm and rotation, as large as the row's largest channel
                err = (codes[at].double() * scale[:, None] - want).abs()
                step = torch.maximum(2.0 ** -4 * want.abs(), scale[:, None] * 2.0 ** -10) * (1 + 2.0 ** -10)
                assert bool((err <= step + 2.0 ** -16 * want.abs().amax(-1, keepdim=True)).all())
            rest = [o for o in range(page) if o not in set(at)]
            ratio = torch.where((kept > 0) & (scale > kept), kept / scale, torch.ones_like(scale)).float()
            assert torch.equal(codes[rest].float(), (old[rest].float() * ratio[:, None]).to(E4M3).float())


@pytest.mark.parametrize("page", [16, 48, 64, 512])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (192, 64)])
def test_runs_with_gaps(page, d, rot):
    # runs of some slots of each page, first from slot 0, then between what is there, with larger values; short runs among
    # many pages, runs of hundreds of tokens, more than a block looks at
    rng, hk, pages = random.Random(page + d), 3, 9
    cache = empty_cache(pages, page, hk, d, d)
    for c in (cache.k, cache.v):
        c.view(torch.uint8)[:] = 0x30
    for turn, scale in enumerate((0.1, 0.1, 40.0, 1.0, 3000.0)):
        runs = {}
        for pg in rng.sample(range(pages), 7):
            at = sorted(rng.sample(range(page), rng.choice([1, 2, page // 3, page - 3])))
            runs[pg] = [0] + [o for o in at if o > 1] if turn == 0 else [o for o in at if o > 0] or [1]
        T = sum(map(len, runs.values()))
        x = write_inputs(80 + turn, T, 4, hk, d, d, rot, True, scale=scale)
        x["kw"] = (x["kw"].float() * scale).bfloat16()
        gaps_check(cache, x, runs)
