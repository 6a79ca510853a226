"""The operators that keep a decoder layer in 8 bits on the GPU -- rms_norm, qk_norm_rope into a PagedCacheFp8,
paged_attention over it -- against plain implementations in 64 bits. Tolerances are derived beside each
comparison. A rounding to e4m3 is off by at most 2^-4 of the value, or half a step of its subnormals, 2^-10."""
import math

import numpy as np
import pytest
import torch

import fp8_block_scaled_fp8bs_gb300 as fp8bs
from test_layer_gpu import gen, no_device_error, norm_rope_close, norm_rope_ref, rand  # noqa: F401

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(a, b):
    return torch.equal(bits(a), bits(b))


def power_above(x):
    """The smallest power of two that is at least x, from the bits (torch.ldexp is not exact on the device)."""
    m, e = torch.frexp(x.double())
    return ((torch.where(m > 0.5, e, e - 1).long() + 1023) << 52).view(torch.float64)


# ---------------------------------------------------------------------------------- rms_norm

def norm_ref(h, w, eps=1e-6):
    h = h.double()
    return h * (h.pow(2).mean(-1, keepdim=True) + eps).rsqrt() * w.double()


def check_norm(got, x, r, w, quant, norm, eps=1e-6):
    # binary32: a sum of squares of at most 64 roundings in a row (all terms positive), the reciprocal root and three
    # products: 2^-17 of the value
    rel = 2.0 ** -17
    h = x
    if r is None:
        assert got.h is None
    else:
        h = (x.float() + r.float()).bfloat16()       # (bf16 numbers: one rounding, whatever holds their sum)
        assert same(got.h, h)
    n = norm_ref(h, w, eps)
    if norm or (norm is None and quant is None):
        assert got.n.dtype == torch.bfloat16
        # (a subnormal step of bf16, where a product is that small)
        assert bool(((got.n.double() - n).abs() <= (2.0 ** -8 + rel) * n.abs() + 2.0 ** -133).all())
    else:
        assert got.n is None
    if quant is None:
        assert got.y is None and got.s is None
        return
    b = n.unflatten(-1, (-1, 128))
    want = b.abs().amax(-1).clamp(min=float(np.float32(1e-4))) / 448
    s = got.s.double()
    if quant == "fp32":
        assert bool(((s - want).abs() <= rel * want).all())
    else:
        assert bool((power_above(got.s) == s).all())
        assert bool((s >= want * (1 - rel)).all()) and bool((s < 2 * want * (1 + rel)).all())
    y = got.y.double().unflatten(-1, (-1, 128))
    step = torch.maximum(2.0 ** -4 * b.abs(), s[..., None] * 2.0 ** -10)
    assert bool(((y * s[..., None] - b).abs() <= step * (1 + 2.0 ** -10) + 2 * rel * b.abs()).all())


@pytest.mark.parametrize("quant,norm", [("fp32", None), ("fp32", True), ("ue8m0", None), (None, None)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,D", [(1, 128), (1, 7168), (3, 256), (5, 384), (200, 1536), (7, 8192), (2, 8320),
                                 (3, 16384), (160, 7168), (500, 640), (1000, 128)])
def test_rms_norm(T, D, residual, quant, norm):
    g = gen(T + D)
    x = rand(g, T, D)
    r = rand(g, T, D, scale=5.0) if residual else None
    w = rand(g, D)
    check_norm(fp8bs.rms_norm(x, w, residual=r, quant=quant, norm=norm), x, r, w, quant, norm)


@pytest.mark.parametrize("quant", ["fp32", "ue8m0"])
def test_rms_norm_sizes_of_values(quant):
    # blocks of zeros, rows of zeros, tiny rows and huge ones, outliers, negative zeros
    g = gen(5)
    x = rand(g, 8, 1024)
    x[0] = 0
    x[1, 128:256] = -0.0
    x[2] *= 1e-30
    x[3] *= 1e15
    x[4, 700] = 30000
    x[5, ::3] = 0
    w = rand(g, 1024)
    w[512:640] = 0
    check_norm(fp8bs.rms_norm(x, w, eps=1e-5, quant=quant, norm=True), x, None, w, quant, True, 1e-5)


def test_rms_norm_strided_and_in_place():
    g = gen(6)
    T, D = 37, 1280
    wide = rand(g, T, D + 264)
    x = wide[:, 8:8 + D]
    r = rand(g, T, D)
    w = rand(g, D)
    ref = fp8bs.rms_norm(x.contiguous(), w, residual=r, quant="fp32", norm=True)
    keep = r.clone()
    got = fp8bs.rms_norm(x, w, residual=r, quant="fp32", norm=True, residual_out=r)
    assert got.h.data_ptr() == r.data_ptr() and all(same(a, b) for a, b in zip(got, ref))
    rw = torch.zeros(T, D + 40, dtype=torch.bfloat16, device="cuda")
    rw[:, 16:16 + D] = keep
    xc = x.contiguous()
    got = fp8bs.rms_norm(xc, w, residual=rw[:, 16:16 + D], quant="fp32", norm=True, residual_out=xc)
    assert got.h.data_ptr() == xc.data_ptr() and all(same(a, b) for a, b in zip(got, ref))
    # each output alone gives the same bits
    assert same(fp8bs.rms_norm(ref.h, w).n, ref.n)
    assert same(fp8bs.rms_norm(ref.h, w, quant="fp32").y, ref.y)


def test_rms_norm_rows_are_independent():
    g = gen(7)
    x = rand(g, 6, 2048)
    w = rand(g, 2048)
    ref = fp8bs.rms_norm(x, w, quant="fp32", norm=True)
    x[2, 5], x[4] = float("nan"), float("inf")
    got = fp8bs.rms_norm(x, w, quant="fp32", norm=True)
    for t in (0, 1, 3, 5):
        assert same(got.n[t], ref.n[t]) and same(got.y[t], ref.y[t]) and same(got.s[t], ref.s[t])
    assert bool(torch.isnan(got.n[2].float()).all())


def test_rms_norm_empty_and_refusals():
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda")
    got = fp8bs.rms_norm(x, w, residual=x, quant="fp32", norm=True)
    assert got.y.shape == (0, 256) and got.s.shape == (0, 2) and got.n.shape == got.h.shape == (0, 256)
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    for kw, error in [(dict(residual=x[:1]), ValueError), (dict(norm=False), ValueError),
                      (dict(quant="int8"), ValueError), (dict(residual_out=x), ValueError),
                      (dict(residual=x.float()), TypeError), (dict(residual=x, residual_out=x[:1]), ValueError)]:
        with pytest.raises(error):
            fp8bs.rms_norm(x, w, **kw)
    with pytest.raises(ValueError):
        fp8bs.rms_norm(x[:, :200], w[:200])
    with pytest.raises(ValueError):
        fp8bs.rms_norm(x, w[:128])
    with pytest.raises(fp8bs.Fp8bsError):                 # over its own rows of another stride
        wide = torch.zeros(2, 512, dtype=torch.bfloat16, device="cuda")
        fp8bs.rms_norm(x, w, residual=wide[:, :256], residual_out=wide.view(-1)[:512].view(2, 256))


def test_rms_norm_feeds_the_product():
    # codes and scales as fp8_gemm takes them: the same product as through act_quant, but for n's own rounding
    g = gen(8)
    x, w = rand(g, 9, 512), rand(g, 512)
    b = (torch.randn(256, 512, generator=g, device="cuda") * 32).to(E4M3)
    bs = torch.full((2, 4), 1 / 512, device="cuda")
    got = fp8bs.rms_norm(x, w, quant="fp32")
    c = fp8bs.fp8_gemm(got.y, got.s, b, bs)
    ref = (got.y.double().unflatten(-1, (4, 128)) * got.s.double()[..., None]).flatten(1) @ (b.double() / 512).T
    assert float((c.double() - ref).abs().max()) <= 2.0 ** -7 * float(ref.abs().max()) + 1e-3 * float(ref.pow(2).mean().sqrt())


# --------------------------------------------------------------------- the write of a cache of codes

def empty_cache(pages, page, hk, dk, dv, order="page-slot-head", seed=1):
    """Codes of any bits (NaN among them) and scales of zero: nothing is held."""
    g = gen(seed)
    def codes(d):
        if order == "page-slot-head":
            return torch.randint(0, 256, (pages, page, hk, d), generator=g, device="cuda", dtype=torch.uint8).view(E4M3)
        return torch.randint(0, 256, (pages, hk, page, d), generator=g, device="cuda", dtype=torch.uint8).view(
            E4M3).transpose(1, 2)
    return fp8bs.PagedCacheFp8(codes(dk), codes(dv), *(torch.zeros(pages, hk, device="cuda") for _ in range(2)))


def copy(cache):
    return fp8bs.PagedCacheFp8(*(t.clone(memory_format=torch.preserve_format) for t in cache))


def write_check(cache, q, k, v, cos, sin, pos, slots, qw=None, kw=None, rot_start=0, interleaved=False):
    """One call against its definition; the cache is changed as the call changed it."""
    before = copy(cache)
    pages, page, hk = cache.k.shape[:3]
    qo = fp8bs.qk_norm_rope(q, k, cos, sin, pos, q_weight=qw, k_weight=kw, rot_start=rot_start,
                            interleaved=interleaved, cache=cache, v=v, slots=slots)
    rq = norm_rope_ref(q, qw, cos, sin, pos, rot_start, interleaved, 1e-6)
    norm_rope_close(qo, rq, float(rq.abs().max()) * 1.5)
    plain = kw is None and cos.shape[1] == 0            # nothing is computed: codes of bf16 numbers, to the bit
    rk = norm_rope_ref(k, kw, cos, sin, pos, rot_start, interleaved, 1e-6)
    at = slots.tolist()
    t = 0
    touched = set()
    while t < len(at):
        if at[t] < 0:
            t += 1
            continue
        pg, off = divmod(at[t], page)
        end = t + 1
        while end < len(at) and at[end] == at[end - 1] + 1 and at[end] // page == pg:
            end += 1
        assert pg not in touched
        touched.add(pg)
        for x, name, exact in ((rk[t:end], "k", plain), (v[t:end].double(), "v", True)):
            codes, scale = getattr(cache, name)[pg], getattr(cache, name + "_scale")[pg].double()
            old, old_scale = getattr(before, name)[pg], getattr(before, name + "_scale")[pg].double()
            need = x.abs().amax((0, 2)).clamp(min=float(np.float32(1e-4))) / 448
            slack = 0.0 if exact else 2.0 ** -17
            kept = torch.where(old_scale > 0, old_scale, torch.zeros_like(old_scale)) if off else torch.zeros_like(need)
            assert bool((power_above(scale) == scale).all())
            # the larger of the old scale and the power of two above `need` (binary32: or the one beside it, where
            # need is within 2^-17 of a power of two; the division by 448 rounds once, 2^-24)
            low = torch.maximum(kept, power_above(need * (1 - slack - 2.0 ** -23)))
            high = torch.maximum(kept, power_above(need * (1 + slack + 2.0 ** -23)))
            assert bool(((scale == low) | (scale == high)).all())
            written = torch.zeros(page, dtype=torch.bool, device="cuda")
            written[off:off + end - t] = True
            if exact:
                assert same(codes[written], (x / scale[:, None]).float().to(E4M3))
            else:
                err = (codes[written].double() * scale[:, None] - x).abs()
                step = torch.maximum(2.0 ** -4 * x.abs(), scale[:, None] * 2.0 ** -10)
                # the rotation's binary32 terms are as large as the row's largest channel
                assert bool((err <= step * (1 + 2.0 ** -10) + 2.0 ** -16 * x.abs().amax(-1, keepdim=True)).all())
            grown = (kept > 0) & (scale > kept)
            ratio = torch.where(grown, kept / scale, torch.ones_like(kept)).float()
            again = (old.float() * ratio[:, None]).to(E4M3)
            want = torch.where(grown[:, None].expand_as(bits(old)), bits(again), bits(old))
            nan = torch.isnan(old.float()) & grown[:, None]              # (of either sign)
            got = bits(codes)
            assert bool(((got == want) | (nan & ((got & 127) == 127)))[~written].all())
        t = end
    rest = [p for p in range(pages) if p not in touched]
    for a, b in zip(cache, before):
        assert same(a[rest], b[rest])
    return qo


def write_inputs(seed, T, hq, hk, dk, dv, rot, norm, scale=1.0):
    g = gen(seed)
    qkv = rand(g, T, hq * dk + hk * dk + hk * dv + 8, scale=scale)
    q = qkv[:, :hq * dk].view(T, hq, dk)
    k = qkv[:, hq * dk:(hq + hk) * dk].view(T, hk, dk)
    v = qkv[:, (hq + hk) * dk:(hq + hk) * dk + hk * dv].view(T, hk, dv)
    ang = torch.rand(4000, rot // 2, generator=g, device="cuda") * 6.28
    pos = torch.randint(0, 4000, (T,), generator=g, device="cuda", dtype=torch.int32)
    w = rand(g, dk) if norm else None
    return dict(q=q, k=k, v=v, cos=ang.cos(), sin=ang.sin(), pos=pos, qw=w, kw=w)


FORMS = [(64, 64, 64, 0, False, True), (64, 64, 32, 16, True, False), (128, 128, 128, 0, False, True),
         (128, 128, 0, 0, False, False), (192, 128, 64, 128, True, False), (256, 64, 128, 64, True, True),
         (16, 32, 16, 0, False, True), (80, 240, 32, 8, False, True)]


@pytest.mark.parametrize("dk,dv,rot,start,interleaved,norm", FORMS)
@pytest.mark.parametrize("order", ["page-slot-head", "page-head-slot"])
@pytest.mark.parametrize("page", [16, 48])
def test_write_runs(dk, dv, rot, start, interleaved, norm, order, page):
    # runs of every kind in one call: a page from its start, its end, its middle, over several pages, single tokens,
    # padding tokens between and inside
    pages, hq, hk = 12, 6, 3
    cache = empty_cache(pages, page, hk, dk, dv, order)
    slots = [*range(5 * page, 7 * page + 3), 3 * page + 15, -1, -5, 9 * page, 2 * page + 7, 2 * page + 8, 4 * page + 1,
             *range(8 * page, 8 * page + 4), 10 * page + page - 1, 11 * page]
    x = write_inputs(page + dk, len(slots), hq, hk, dk, dv, rot, norm)
    kw = dict(rot_start=start, interleaved=interleaved)
    write_check(cache, slots=torch.tensor(slots, device="cuda"), **x, **kw)
    # the same pages go on: smaller values leave the scales, larger ones of some heads raise them
    more = [7 * page + 3, 7 * page + 4, 9 * page + 1, *range(8 * page + 4, 8 * page + 16), 2 * page + 9, 11 * page + 1]
    y = write_inputs(page + dk + 1, len(more), hq, hk, dk, dv, rot, norm, scale=0.1)
    write_check(cache, slots=torch.tensor(more, device="cuda"), **y, **kw)
    last = [7 * page + 5, 9 * page + 2, 2 * page + 10, 11 * page + 2]
    z = write_inputs(page + dk + 2, len(last), hq, hk, dk, dv, rot, norm)
    z["k"][:, 1] *= 64
    z["v"][:, 2] *= 300
    z["v"][1] = 0
    write_check(cache, slots=torch.tensor(last, device="cuda"), **z, **kw)
    # and pages begin anew, whatever their scales were
    anew = [9 * page, 9 * page + 1, 2 * page]
    u = write_inputs(page + dk + 3, len(anew), hq, hk, dk, dv, rot, norm, scale=1e-3)
    write_check(cache, slots=torch.tensor(anew, device="cuda"), **u, **kw)


@pytest.mark.parametrize("T,page", [(1, 16), (127, 16), (130, 128), (300, 512), (2047, 64), (2048, 64), (2500, 48),
                                    (5000, 1024)])
@pytest.mark.parametrize("off", [0, 5])
def test_write_chunks(T, page, off):
    pages = (T + off) // page + 3
    cache = empty_cache(pages, page, 2, 128, 128)
    x = write_inputs(T, T, 3, 2, 128, 128, 128, True)
    write_check(cache, slots=torch.arange(off + page, off + page + T, device="cuda"), **x)


@pytest.mark.parametrize("dk,dv,rot", [(64, 64, 64), (128, 128, 128), (192, 128, 64)])
@pytest.mark.parametrize("T,page", [(511, 512), (512, 80), (700, 512)])
@pytest.mark.parametrize("heads", [1, 5])
def test_write_windows(dk, dv, rot, T, page, heads):
    # runs longer than what a block keeps, and those that end in the next block's tokens, in pages that are held in
    # part and whose scales grow; tables of cosines at odd addresses
    off = 37
    pages = (T + off) // page + 3
    cache = empty_cache(pages, page, heads, dk, dv)
    x = write_inputs(T + heads, off, heads, heads, dk, dv, rot, True, scale=0.01)
    write_check(cache, slots=torch.arange(page, page + off, device="cuda"), **x)
    x = write_inputs(T, T, 2 * heads, heads, dk, dv, rot, True)
    for name in ("cos", "sin"):
        odd = torch.empty(x[name].numel() + 1, device="cuda")
        odd[1:] = x[name].flatten()
        x[name] = odd[1:].view(x[name].shape)
    write_check(cache, slots=torch.arange(off + page, off + page + T, device="cuda"), **x)


def test_write_chunk_of_many_sequences():
    # 2048 tokens and more: runs that begin anywhere among the tokens that one block looks at
    page, hk = 16, 2
    g = gen(3)
    need = [int(n) for n in torch.randint(1, 40, (200,), generator=g, device="cuda")]
    slots, at = [], page
    for i, n in enumerate(need):
        off = (i * 5) % page if i % 3 else 0
        slots += list(range(at + off, at + off + n)) + ([-1] if i % 7 == 0 else [])
        at += -(-(off + n) // page) * page
    cache = empty_cache(at // page + 1, page, hk, 64, 64)
    assert len(slots) > 2048
    x = write_inputs(4, len(slots), 2, hk, 64, 64, 64, True)
    write_check(cache, slots=torch.tensor(slots, device="cuda"), **x)


def test_write_token_by_token():
    # a page filled by single tokens holds what it can: each code within half a step of the final scale, and half a
    # subnormal step of it for each time that the scale grew (at most the number of doublings)
    page, hk, d = 32, 2, 128
    cache = empty_cache(2, page, hk, d, d)
    x = write_inputs(9, page, 2, hk, d, d, 128, True)
    x["v"] *= torch.logspace(-3, 3, page, device="cuda").bfloat16()[:, None, None]
    for t in range(page):
        write_check(cache, slots=torch.tensor([page + t], device="cuda"),
                    **{n: (a[t:t + 1] if n in ("q", "k", "v", "pos") else a) for n, a in x.items()})
    s = cache.v_scale[1].double()
    whole = copy(cache)
    write_check(whole, slots=torch.arange(page, 2 * page, device="cuda"), **x)
    assert same(whole.k_scale[1], cache.k_scale[1]) and same(whole.v_scale[1], cache.v_scale[1])
    err = (cache.v[1].double() * s[:, None] - x["v"].double()).abs()
    assert bool((err <= torch.maximum(2.0 ** -4 * x["v"].double().abs(), 21 * s[:, None] * 2.0 ** -10)).all())


def test_write_values_that_are_not_finite():
    page, hk, d = 16, 2, 64
    cache = empty_cache(3, page, hk, d, d)
    x = write_inputs(10, 4, 2, hk, d, d, 0, False)
    x["k"][1, 0, 5], x["v"][2, 1, 7], x["v"][0, 0, 3] = float("nan"), float("inf"), -float("inf")
    fp8bs.qk_norm_rope(x["q"], x["k"], x["cos"], x["sin"], x["pos"], cache=cache, v=x["v"],
                       slots=torch.arange(page, page + 4, device="cuda"))
    assert bool(torch.isnan(cache.k[1, 1, 0, 5].float())) and int(torch.isnan(cache.k[1, :4].float()).sum()) == 1
    assert float(cache.v[1, 2, 1, 7]) == 448 and float(cache.v[1, 0, 0, 3]) == -448
    assert bool(torch.isfinite(cache.v_scale).all()) and not bool(torch.isnan(cache.v[1, :4].float()).any())
    assert same(cache.k[1, :4, 1], (x["k"][:, 1].float() / cache.k_scale[1, 1]).to(E4M3))


def test_write_reports_bad_indices():
    page, hk, d = 16, 1, 64
    cache = empty_cache(2, page, hk, d, d)
    before = copy(cache)
    x = write_inputs(11, 5, 2, hk, d, d, 32, True)
    x["pos"][:] = torch.tensor([1, 4000, 2, -1, 3], device="cuda")
    slots = torch.tensor([2 * page, 3, 4, 5, 1 << 40], device="cuda")
    qo = fp8bs.qk_norm_rope(x["q"], x["k"], x["cos"], x["sin"], x["pos"], q_weight=x["qw"], k_weight=x["kw"],
                            cache=cache, v=x["v"], slots=slots)
    assert fp8bs.fp8bs_device_error(clear=True) == fp8bs.DEVERR_INDEX
    assert bool((qo[[1, 3]] == 0).all()) and not bool((qo[[0, 2, 4]] == 0).all())
    for a, b in ((cache.k, before.k), (cache.v, before.v)):
        assert same(a[0, :4], b[0, :4]) and same(a[0, 5:], b[0, 5:]) and same(a[1], b[1])
    assert same(cache.v[0, 4], (x["v"][2].float() / cache.v_scale[0, 0]).to(E4M3))
    assert float(cache.k_scale[1, 0]) == 0


def test_write_far_slots():
    # codes past 2^32 bytes
    pages, page, hk, d = 80000, 64, 8, 128
    cache = fp8bs.PagedCacheFp8(*(torch.empty(pages, page, hk, d, dtype=E4M3, device="cuda") for _ in range(2)),
                                *(torch.zeros(pages, hk, device="cuda") for _ in range(2)))
    x = write_inputs(12, 3, 8, hk, d, d, 0, False)
    slots = torch.tensor([pages * page - 1, (2 ** 32 // (hk * d)) + 5, 0], device="cuda")
    fp8bs.qk_norm_rope(x["q"], x["k"], x["cos"], x["sin"], x["pos"], cache=cache, v=x["v"], slots=slots)
    for t, s in enumerate(slots.tolist()):
        for rows, codes, scale in ((x["k"], cache.k, cache.k_scale), (x["v"], cache.v, cache.v_scale)):
            sc = scale[s // page]
            assert bool((sc > 0).all())
            assert same(codes[s // page, s % page], (rows[t].float() / sc[:, None]).to(E4M3))


def test_cache_refusals():
    x = write_inputs(13, 2, 2, 2, 64, 64, 64, True)
    slots = torch.arange(2, device="cuda")

    def write(cache, **kw):
        fp8bs.qk_norm_rope(x["q"], x["k"], x["cos"], x["sin"], x["pos"], cache=cache,
                           **{**dict(v=x["v"], slots=slots), **kw})

    c = empty_cache(2, 16, 2, 64, 64)
    with pytest.raises(ValueError):
        write(c._replace(k_scale=c.k_scale[:1]))
    with pytest.raises(ValueError):
        write(c._replace(v_scale=torch.zeros(2, 4, device="cuda")[:, ::2]))
    with pytest.raises(TypeError):
        write(c._replace(v_scale=c.v_scale.double()))
    with pytest.raises(TypeError):
        write(c._replace(k=c.k.view(torch.uint8)))
    with pytest.raises(TypeError):
        write(c[:3])
    with pytest.raises(TypeError):
        write(fp8bs.PagedCache(c.k, c.v))
    with pytest.raises(ValueError):
        write(c, slots=None)
    with pytest.raises(ValueError):
        write(empty_cache(2, 16, 3, 64, 64))
    with pytest.raises(fp8bs.Fp8bsError):
        write(empty_cache(2, 24, 2, 64, 64))                 # pages of 24 slots
    q = rand(gen(1), 1, 2, 64)
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    with pytest.raises(fp8bs.Fp8bsError):
        fp8bs.paged_attention(q, empty_cache(2, 8, 2, 64, 64), table, start, one)
    with pytest.raises(fp8bs.Fp8bsError):
        fp8bs.paged_attention(q, empty_cache(2, 16, 2, 64, 128), table, start, one)
    with pytest.raises(ValueError):
        fp8bs.paged_attention(q, empty_cache(2, 16, 2, 128, 128), table, start, one)


# ------------------------------------------------------------------- attention over a cache of codes

def fp8_case(seed, news, lens, hq, hk, dk, dv, page, order="page-slot-head", spare=3, poison=True, q_scale=1.0,
             k_spread=1.0, v_spread=4.0):
    """Random codes; scales that differ from page to page and head to head by 2^+-spread. Codes outside the keys are
    NaN, the scales of pages without keys any numbers, table entries past the keys outside the cache."""
    g = gen(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    def codes(d):
        shape = (pages, page, hk, d) if order == "page-slot-head" else (pages, hk, page, d)
        c = (torch.randn(shape, generator=g, device="cuda") * 100).clamp(-448, 448).to(E4M3)
        return c if order == "page-slot-head" else c.transpose(1, 2)
    def scales(spread, mean):
        e = torch.rand(pages, hk, generator=g, device="cuda") * (2 * spread) - spread
        return torch.exp2(e.round() + mean)
    k, v, ks, vs = codes(dk), codes(dv), scales(k_spread, -7), scales(v_spread, -7)
    perm = torch.randperm(pages, generator=g, device="cuda").tolist()
    table = torch.full((len(lens), max(need + [1]) + 1), -7, dtype=torch.int32)
    used = torch.zeros(pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(need[b]):
            table[b, j] = perm.pop()
            used[table[b, j], :min(page, n - j * page)] = True
    if poison:
        k.view(torch.uint8)[~used.cuda()] = 0x7F
        v.view(torch.uint8)[~used.cuda()] = 0xFF
        ks[perm] = float("nan")
        vs[perm] = -1.0
    q = rand(g, sum(news), hq, dk, scale=q_scale)
    starts = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32, device="cuda")
    return dict(q=q, cache=fp8bs.PagedCacheFp8(k, v, ks, vs), page_table=table.cuda(), q_start=starts,
                kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def held(c, b, L):
    """Keys and values [L, heads, d] of sequence b, their codes' values and scales, in 64 bits."""
    cache = c["cache"]
    page = cache.k.shape[1]
    j = torch.arange(L, device="cuda")
    pg = c["page_table"][b].long()[j // page]
    take = lambda x: x.view(torch.uint8)[pg, j % page].view(E4M3).double()  # noqa: E731
    ks, vs = cache.k_scale.double()[pg], cache.v_scale.double()[pg]
    return take(cache.k) * ks[..., None], take(cache.v), vs


def fp8_ref(c, news, lens, scale, causal, window):
    """(o, lse, bound of o's error, bound of lse's error) in 64 bits.

    Scores: q is held in two e4m3 pieces whose sum is q to 2^-10 of a unit in which q's largest channel is at least 224
    (2^-17 of that channel); the sum over 192 channels is binary32, 2^-16 of its terms at most. With z the largest error
    of a score, every p is within 2 z of its value, lse within z.
    Probabilities, times their value's scale and relative to the largest such product in reach: one rounding to bf16, or
    two e4m3 pieces: 2^-8 of p, and 2^-23 of the largest p vs for each code where p vanishes beside it.
    The output: 2^-8 of |o| <= sum p |v|. Exponentials and binary32 sums: 2^-12 of the sum covers them."""
    q = c["q"]
    T, hq, dk = q.shape
    hk, dv = c["cache"].v.shape[2:]
    grp = hq // hk
    o = torch.zeros(T, hq, dv, dtype=torch.float64, device="cuda")
    far = torch.zeros_like(o)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device="cuda")
    off = torch.zeros(T, hq, dtype=torch.float64, device="cuda")
    t = 0
    for b, (n, L) in enumerate(zip(news, lens)):
        if n and L:
            k, v, vs = held(c, b, L)
            i = torch.arange(n, device="cuda")[:, None]
            j = torch.arange(L, device="cuda")
            seen = (j <= L - n + i) if causal else torch.ones(n, L, dtype=torch.bool, device="cuda")
            if window:
                seen &= j > L - n + i - window
            for h in range(hq):
                kh = h // grp
                qd = q[t:t + n, h].double()
                s = (qd @ k[:, kh].T * scale).masked_fill(~seen, -math.inf)
                l = torch.logsumexp(s, 1)
                lse[t:t + n, h] = l
                p = torch.exp(s - l[:, None]).nan_to_num(0.0)
                vv = v[:, kh] * vs[:, kh, None]
                o[t:t + n, h] = p @ vv
                mag = p @ vv.abs()
                size = qd.abs().amax(1) * (k[:, kh].abs().sum(1)[None] * seen).amax(1) * abs(scale)
                z = size * (2.0 ** -17 + 2.0 ** -16) + 2.0 ** -20 * l.abs().nan_to_num(0, 0, 0)
                top = (p * vs[:, kh]).amax(1)
                floor = 2.0 ** -23 * top[:, None] * (seen.double() @ v[:, kh].abs())
                far[t:t + n, h] = (2.0 ** -7 + 2.0 ** -12 + 2 * z[:, None]) * mag + floor + 1e-30
                off[t:t + n, h] = z + 1e-5
        t += n
    return o, lse, far, off


def fp8_check(c, news, lens, scale=None, causal=True, window=0, **kw):
    T, hq, dk = c["q"].shape
    dv = c["cache"].v.shape[3]
    guard = torch.full((T + 2, hq, dv), 3.0, dtype=torch.bfloat16, device="cuda")
    out, lse = fp8bs.paged_attention(**c, scale=scale, causal=causal, window=window, return_lse=True,
                                     out=guard[1:T + 1], **kw)
    o, l, far, off = fp8_ref(c, news, lens, dk ** -0.5 if scale is None else scale, causal, window)
    assert bool((guard[0] == 3).all()) and bool((guard[T + 1] == 3).all())
    err = (out.double() - o).abs()
    assert bool((err <= far).all()), float((err / far).nan_to_num(math.inf).max())
    empty = torch.isinf(l)
    assert bool((out[empty] == 0).all())
    assert torch.equal(torch.isinf(lse), empty) and bool((lse[empty] < 0).all())
    wrong = (lse.double() - l).abs()[~empty]
    assert bool((wrong <= off[~empty]).all()), float((wrong / off[~empty]).max())
    return out, lse


SHAPES = [(64, 64), (128, 128), (192, 128)]


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (8, 1), (7, 1), (6, 2), (32, 4), (16, 1), (24, 1), (40, 1), (128, 1)])
def test_decode(dk, dv, hq, hk):
    lens = [1, 2, 63, 64, 65, 127, 128, 129, 300, 1000]
    news = [1] * len(lens)
    fp8_check(fp8_case(1, news, lens, hq, hk, dk, dv, 16), news, lens)


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("news,lens", [
    ([128], [128]), ([1], [1]), ([129], [129]), ([200], [333]), ([64, 1, 0, 17], [64, 500, 30, 17]),
    ([300, 5], [300, 1029]), ([2, 2, 2], [2, 130, 257]), ([3, 8, 9, 1], [700, 8, 900, 130]),
])
@pytest.mark.parametrize("hq,hk", [(4, 4), (4, 1), (6, 2)])
def test_chunks(dk, dv, news, lens, hq, hk):
    fp8_check(fp8_case(2, news, lens, hq, hk, dk, dv, 32), news, lens)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 192, 208, 256, 512])
@pytest.mark.parametrize("order", ["page-slot-head", "page-head-slot"])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_page_sizes(page, order, dk, dv):
    for news, lens in (([1, 4, 3], [517, 200, 3]), ([1, 140, 3], [517, 200, 3])):
        fp8_check(fp8_case(3, news, lens, 8, 2, dk, dv, page, order), news, lens)


@pytest.mark.parametrize("window", [1, 2, 100, 128, 5000, 2 ** 62])
@pytest.mark.parametrize("hq,hk", [(4, 4), (8, 1)])
def test_window(window, hq, hk):
    for news, lens in (([1, 1, 1, 0, 2], [1000, 400, 1, 9, 777]), ([1, 150, 1, 0, 20], [1000, 400, 1, 9, 777])):
        fp8_check(fp8_case(4, news, lens, hq, hk, 64, 64, 16), news, lens, window=window)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("T", [1, 20, 200])
def test_window_over_freed_pages(page, T):
    news, lens, window = [T, 1], [1500, 700], 150
    c = fp8_case(16, news, lens, 4, 2, 128, 128, page)
    ref = fp8bs.paged_attention(**c, window=window, return_lse=True)
    for b, (n, L) in enumerate(zip(news, lens)):
        gone = max(0, L - n - window + 1) // page
        there = c["page_table"][b, :gone].long()
        c["cache"].k.view(torch.uint8)[there] = 0x7F
        c["cache"].v.view(torch.uint8)[there] = 0x7F
        c["cache"].k_scale[there] = float("nan")
        c["cache"].v_scale[there] = float("nan")
        c["page_table"][b, :gone] = -1
    out = fp8bs.paged_attention(**c, window=window, return_lse=True)
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    assert bool(torch.isfinite(out[0].float()).all())


@pytest.mark.parametrize("news", [[1, 1, 3], [1, 1, 90]])
def test_reports_bad_lengths(news):
    lens = [100, 60, 140]
    c = fp8_case(17, news, lens, 4, 2, 64, 64, 16)
    ref = fp8bs.paged_attention(**c)
    c["kv_len"][1] = 10 ** 6
    out = fp8bs.paged_attention(**c)
    assert fp8bs.fp8bs_device_error(clear=True) == fp8bs.DEVERR_INDEX
    assert torch.equal(out[0], ref[0]) and torch.equal(out[2:], ref[2:])


@pytest.mark.parametrize("bad", [-1, 1 << 30])
@pytest.mark.parametrize("news", [[1, 1], [1, 150]])
def test_pages_outside_the_cache_read_as_zeros(news, bad):
    lens = [300, 400]
    c = fp8_case(21, news, lens, 8, 2, 128, 128, 64, poison=False)
    at = int(c["page_table"][1, 2])
    c["page_table"][1, 2] = bad
    out = fp8bs.paged_attention(**c, return_lse=True)
    assert fp8bs.fp8bs_device_error(clear=True) == fp8bs.DEVERR_INDEX
    c["page_table"][1, 2] = at
    c["cache"].k.view(torch.uint8)[at] = 0
    c["cache"].v.view(torch.uint8)[at] = 0
    o, l, far, off = fp8_ref(c, news, lens, 128 ** -0.5, True, 0)
    assert bool(((out[0].double() - o).abs() <= far).all()) and bool(((out[1].double() - l).abs() <= off).all())


@pytest.mark.parametrize("B", [257, 700])
def test_many_sequences(B):
    news = [(b * 7) % 4 for b in range(B)]
    lens = [max(n, (b * 13) % 90) for b, n in enumerate(news)]
    fp8_check(fp8_case(18, news, lens, 2, 1, 64, 64, 16), news, lens)


@pytest.mark.parametrize("window", [0, 50])
def test_not_causal(window):
    for news, lens in (([7, 2, 1], [300, 130, 0]), ([7, 130, 1], [300, 130, 0])):
        fp8_check(fp8_case(5, news, lens, 4, 2, 128, 128, 16), news, lens, causal=False, window=window)


def test_rows_without_keys():
    for news, lens in (([10, 3, 2], [4, 0, 60]), ([10, 3, 200], [4, 0, 60])):
        out, lse = fp8_check(fp8_case(6, news, lens, 4, 2, 128, 128, 16), news, lens)
        assert bool(torch.isinf(lse[:6]).all()) and bool(torch.isinf(lse[10:13]).all())


@pytest.mark.parametrize("T,L,hq,hk", [(1, 20000, 8, 1), (1, 9999, 2, 2), (4, 12345, 8, 2), (1, 33000, 16, 2)])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_long_keys(T, L, hq, hk, dk, dv):
    fp8_check(fp8_case(7, [T], [L], hq, hk, dk, dv, 64), [T], [L])


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("n,L,hq,hk,window,causal", [
    (700, 1700, 8, 2, 0, True), (1999, 2300, 24, 8, 0, True), (1230, 3001, 8, 4, 500, True),
    (1230, 1300, 4, 2, 0, False),
])
def test_long_chunks(dk, dv, n, L, hq, hk, window, causal):
    fp8_check(fp8_case(17, [n], [L], hq, hk, dk, dv, 32), [n], [L], window=window, causal=causal)


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("hq,hk", [(16, 16), (32, 4)])
def test_mixed_batch(dk, dv, hq, hk):
    news, lens = [700, 1, 1, 300, 2, 0, 1, 16], [700, 900, 3000, 2001, 40, 9, 1, 16]
    fp8_check(fp8_case(18, news, lens, hq, hk, dk, dv, 16), news, lens)


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("hq,hk", [(3, 3), (8, 1), (24, 2), (24, 1), (40, 1)])
def test_mixed_batch_of_every_row_form(dk, dv, hq, hk):
    # single tokens beside a chunk: those of the chunk's kernel, and few of either side of what the other takes
    news, lens = [130, 1, 3, 8, 9, 1, 33, 0], [200, 700, 40, 300, 9, 1, 1100, 5]
    fp8_check(fp8_case(31, news, lens, hq, hk, dk, dv, 16), news, lens, max_q_len=130, max_kv_len=1100)


@pytest.mark.parametrize("news,most", [([1, 40], 40), ([3, 0, 1], 50), ([1, 1], 2), ([7, 7], 40)])
@pytest.mark.parametrize("hq,hk", [(4, 4), (8, 1), (40, 1)])
def test_padded_batches(news, most, hq, hk):
    # as many rows as sequences of the largest length would have; those behind the last sequence stay as they were
    lens = [n + 100 for n in news]
    c = fp8_case(32, news, lens, hq, hk, 128, 128, 16)
    T, rows = len(news) * most, sum(news)
    out = torch.full((T, hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    o, l, far, off = fp8_ref(c, news, lens, 128 ** -0.5, True, 0)
    q = torch.full((T, hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[:rows] = c["q"]
    got, lse = fp8bs.paged_attention(**{**c, "q": q}, out=out, return_lse=True, max_q_len=most, max_kv_len=max(lens))
    assert bool(((got[:rows].double() - o).abs() <= far).all())
    assert bool(((lse[:rows].double() - l).abs() <= off).all())
    assert bool((got[rows:] == 3).all())


@pytest.mark.parametrize("scale", [0.0, 1.0, 3.0, -0.125])
def test_scales(scale):
    for news, lens in (([1, 1], [600, 700]), ([1, 130], [600, 700])):
        fp8_check(fp8_case(9, news, lens, 4, 2, 64, 64, 16, k_spread=0), news, lens, scale=scale)


@pytest.mark.parametrize("k_spread,v_spread", [(0, 20), (6, 0), (0, 60)])
def test_pages_of_very_different_scales(k_spread, v_spread):
    # (the page with the largest products decides what the output can resolve)
    for news, lens in (([1, 2], [6000, 700]), ([1, 130], [600, 700])):
        fp8_check(fp8_case(12, news, lens, 4, 2, 128, 128, 16, k_spread=k_spread, v_spread=v_spread), news, lens,
                  scale=0.01)


def test_a_sink_and_a_long_tail():
    # one key takes most of the weight while its value is small; all others share the rest in equal parts
    L, hk, d = 16000, 1, 128
    c = fp8_case(13, [1], [L], 4, hk, d, d, 16, k_spread=0, v_spread=0)
    k = c["cache"].k.view(torch.uint8)
    k[:] = torch.ones(1, device="cuda").to(E4M3).view(torch.uint8)
    first = int(c["page_table"][0, 0])
    k[first, 0] = torch.full((1,), 3.0, device="cuda").to(E4M3).view(torch.uint8)
    c["cache"].k_scale.fill_(1.0)
    c["q"].fill_(1.0)
    c["cache"].v_scale[first] *= 2.0 ** -9
    for scale in (0.03125, 0.0390625, 0.0625):             # the sink: 2^11.5, 2^14.4 and 2^23 times another key
        fp8_check(c, [1], [L], scale=scale)


def test_strided_queries_and_tight_bounds():
    for n in (5, 70):
        news, lens = [n, 1], [90, 333]
        c = fp8_case(10, news, lens, 4, 2, 128, 128, 16)
        wide = torch.zeros(n + 1, 9, 128, dtype=torch.bfloat16, device="cuda")
        wide[:, 3:7] = c["q"]
        c["q"] = wide[:, 3:7]
        fp8_check(c, news, lens, max_q_len=n, max_kv_len=333)


@pytest.mark.parametrize("size", [1e-30, 1e-8, 1e8, 1e25])
def test_sizes_of_queries(size):
    # queries and keys whose sizes cancel, rows of very different size, channels far out, a row of zeros
    for news, lens in (([1, 3], [500, 200]), ([1, 130], [500, 200])):
        c = fp8_case(14, news, lens, 8, 2, 128, 128, 16)
        c["q"][:, 1] *= 16
        c["q"][:, 3] *= 1 / 64
        c["q"][:, 4, ::17] *= 100
        c["q"][:, 5] = 0
        c["q"] = (c["q"].float() * size).bfloat16()
        fp8_check(c, news, lens, scale=128 ** -0.5 / size / 8)


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("n,L", [(1, 40), (1, 20000), (5, 3000), (300, 400)])
def test_scores_that_are_not_finite(dk, dv, n, L):
    c = fp8_case(15, [n], [L], 8, 2, dk, dv, 16, spare=0, poison=False)
    ref, lref = fp8bs.paged_attention(**c, return_lse=True)
    c["q"][0, 0, 3] = float("nan")
    c["q"][0, 1, dk - 1] = float("inf")
    at = (L - 1) // 16
    c["cache"].k.view(torch.uint8)[int(c["page_table"][0, at]), (L - 1) % 16, 1, 5] = 0x7F
    out, lse = fp8bs.paged_attention(**c, return_lse=True)
    bad = torch.zeros(n, 8, dtype=torch.bool, device="cuda")
    bad[0, :2] = True
    bad[n - 1, 4:] = True                                   # the last key is seen by the last query alone
    assert bool(torch.isnan(out[bad].float()).all()) and bool(torch.isnan(lse[bad]).all())
    assert torch.equal(out[~bad], ref[~bad]) and torch.equal(lse[~bad], lref[~bad])


@pytest.mark.parametrize("n,L", [(1, 40), (1, 20000), (300, 400)])
def test_a_scale_that_is_not_a_number(n, L):
    c = fp8_case(19, [n], [L], 8, 2, 128, 128, 16)
    out, lse = fp8bs.paged_attention(**c, scale=float("nan"), return_lse=True)
    assert bool(torch.isnan(out.float()).all()) and bool(torch.isnan(lse).all())


def test_same_bits_twice_and_on_another_stream():
    news, lens = [1, 1, 30], [5000, 77, 800]
    c = fp8_case(11, news, lens, 8, 2, 128, 128, 16)
    a = fp8bs.paged_attention(**c, return_lse=True)
    b = fp8bs.paged_attention(**c, return_lse=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        d = fp8bs.paged_attention(**c, return_lse=True)
    s.synchronize()
    for x, y, z in zip(a, b, d):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_far_pages():
    # codes past 2^32 bytes
    pages, page, hk, d = 70000, 64, 8, 128
    k, v = (torch.empty(pages, page, hk, d, dtype=E4M3, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(pages, hk, device="cuda") / 128 for _ in range(2))
    g = gen(20)
    table = torch.tensor([[pages - 1, 0, 65540, 5]], dtype=torch.int32, device="cuda")
    for p in table[0].tolist():
        for x in (k, v):
            x[p] = (torch.randn(page, hk, d, generator=g, device="cuda") * 100).clamp(-448, 448).to(E4M3)
    for n in (1, 100):
        c = dict(q=rand(g, n, 16, d), cache=fp8bs.PagedCacheFp8(k, v, ks, vs), page_table=table,
                 q_start=torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                 kv_len=torch.tensor([250], dtype=torch.int32, device="cuda"))
        fp8_check(c, [n], [250])


def test_tables_far_wider_than_the_sequences():
    for news, lens in (([1] * 30, [10 * b + 1 for b in range(30)]), ([500, 1], [500, 3000])):
        c = fp8_case(22, news, lens, 64, 8, 64, 64, 16)
        wide = torch.full((len(lens), 1 << 18), -7, dtype=torch.int32, device="cuda")
        wide[:, :c["page_table"].shape[1]] = c["page_table"]
        c["page_table"] = wide
        fp8_check(c, news, lens)


# ------------------------------------------------------------------------------------- together

def layer_steps(cache, steps, x, w, out):
    """Norm, write and attention of several steps of two sequences, as a layer runs them; the outputs into `out`."""
    page = cache.k.shape[1]
    hk, d = cache.k.shape[2:]
    hq = 2 * hk
    table = torch.arange(cache.k.shape[0], dtype=torch.int32, device="cuda").view(2, -1)
    ang = torch.arange(512, device="cuda")[:, None] * torch.rand(d // 2, device="cuda", generator=gen(2))
    cos, sin = ang.cos(), ang.sin()
    lens = [0, 0]
    made = []
    for new in steps:
        T = sum(new)
        at = [(b, lens[b] + i) for b in range(2) for i in range(new[b])]
        lens = [a + n for a, n in zip(lens, new)]
        made.append((T, torch.tensor([int(table[b, j // page]) * page + j % page for b, j in at], device="cuda"),
                     torch.tensor([j for _, j in at], dtype=torch.int32, device="cuda"),
                     torch.tensor([0, new[0], T], dtype=torch.int32, device="cuda"),
                     torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens)))

    def run():
        t = 0
        for T, slots, pos, starts, kv, most in made:
            got = fp8bs.rms_norm(x[t:t + T], w, quant="fp32", norm=True)
            qkv = got.n[:, :(hq + 2 * hk) * d]
            q, k, v = (z.unflatten(1, (-1, d)) for z in qkv.split([hq * d, hk * d, hk * d], 1))
            q = fp8bs.qk_norm_rope(q, k, cos, sin, pos, cache=cache, v=v, slots=slots)
            out[t:t + T] = fp8bs.paged_attention(q, cache, table, starts, kv, max_kv_len=most).flatten(1)
            t += T
    return run


@pytest.mark.parametrize("capture", [False, True])
def test_steps_of_a_layer(capture):
    # chunks, single tokens and both; eager, and captured and replayed on other contents
    hk, d, page = 2, 128, 16
    steps = [[40, 3], [1, 1], [1, 70], [5, 1], [1, 1]]
    T = sum(map(sum, steps))
    g = gen(30)
    x, w = rand(g, T, 1024), rand(g, 1024)
    cache = empty_cache(24, page, hk, d, d)
    fresh = copy(cache)
    out = torch.zeros(T, 2 * hk * d, dtype=torch.bfloat16, device="cuda")
    run = layer_steps(cache, steps, x, w, out)
    run()
    ref = out.clone()
    # against the layer in 64 bits, from the cache as it was written
    assert bool(torch.isfinite(ref.float()).all()) and float(ref.float().abs().max()) > 0
    if capture:
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            run()
        for a, b in zip(cache, fresh):
            a.copy_(b)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, ref)
        y = rand(g, T, 1024)
        x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        again = out.clone()
        out.zero_()
        run()
        assert same(out, again) and not same(out, ref)


def test_cache_of_codes_beside_a_bf16_cache():
    # the same tokens into both caches: the outputs differ by the codes' rounding of keys and values alone. A value is
    # 2^-4 of itself off at most (2^-5 on average over a binade), a score sums 128 such errors of either sign:
    # 2^-4 |q||k| / sqrt(128) sqrt(d) scale, some hundredths, so p moves by hundredths; a tenth of the size covers both.
    g = gen(31)
    T, hq, hk, d, page = 200, 8, 2, 128, 16
    q, k, v = rand(g, T, hq, d), rand(g, T, hk, d), rand(g, T, hk, d)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    ang = torch.arange(T, device="cuda")[:, None] * torch.rand(d // 2, device="cuda", generator=g)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    slots = torch.arange(T, device="cuda")
    table = torch.arange(13, dtype=torch.int32, device="cuda")[None]
    start = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    kv = torch.tensor([T], dtype=torch.int32, device="cuda")
    outs = []
    for cache in (fp8bs.PagedCache(*(torch.zeros(13, page, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))),
                  empty_cache(13, page, hk, d, d)):
        qr = fp8bs.qk_norm_rope(q, k, ang.cos(), ang.sin(), pos, q_weight=w, k_weight=w, cache=cache, v=v, slots=slots)
        outs.append((qr, fp8bs.paged_attention(qr, cache, table, start, kv).double()))
    assert same(outs[0][0], outs[1][0])
    assert float((outs[0][1] - outs[1][1]).norm() / outs[0][1].norm()) < 0.1


def attention_call(seed):
    c = fp8_case(seed, [1, 1], [9000, 5000], 16, 4, 128, 128, 16)
    return lambda: fp8bs.paged_attention(**c)


def chunk_call(seed):
    c = fp8_case(seed, [200, 1], [900, 5000], 16, 4, 128, 128, 16)
    return lambda: fp8bs.paged_attention(**c)


@pytest.mark.parametrize("call", [attention_call, chunk_call])
def test_graphs_of_one_capture_stream_in_flight_at_once(call):
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
    for _ in range(30):
        eager = []
        for _ in range(4):
            for s, graph in zip(side, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
            with torch.cuda.stream(capture):
                eager.append(calls[1]())
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for o, r in zip(outs, refs)) and all(torch.equal(o, refs[1]) for o in eager)


def narrow_call(seed):
    c = fp8_case(seed, [30, 1, 1], [9000, 5000, 40], 16, 4, 128, 128, 16)
    return lambda: fp8bs.paged_attention(**c, max_q_len=30, max_kv_len=9000)


def test_graphs_of_short_chunks_in_flight_at_once():
    test_graphs_of_one_capture_stream_in_flight_at_once(narrow_call)


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("chunks", [{5: 40, 70: 300, 149: 33}, {149: 400}, {0: 20, 63: 20, 64: 20, 128: 20}])
def test_chunks_among_many_sequences(dk, dv, chunks):
    # more sequences than are looked through at once, some out of order in length, some without tokens
    news = [chunks.get(b, 0 if b % 11 == 3 else 1) for b in range(150)]
    lens = [n + 7 * b % 500 for b, n in enumerate(news)]
    fp8_check(fp8_case(33, news, lens, 8, 2, dk, dv, 16), news, lens, max_q_len=max(news), max_kv_len=max(lens))
