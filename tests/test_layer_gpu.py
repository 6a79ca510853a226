"""The operators around the FP8 products of a decoder layer on the GPU, against plain implementations
in 64 bits. Tolerances are derived beside each comparison."""
import math

import numpy as np
import pytest
import torch

import fp8_block_scaled_fp8bs_gb300 as fp8bs

pytestmark = pytest.mark.gpu

ULP = 2.0 ** -7          # spacing of bf16 (8 significant bits) relative to the value, at most; its
                         # rounding is half of it


@pytest.fixture(autouse=True)
def no_device_error():
    fp8bs.fp8bs_device_error(clear=True)
    yield
    assert fp8bs.fp8bs_device_error(clear=True) == 0


def rand(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------------------ qk_norm_rope

def norm_rope_ref(x, w, cos, sin, pos, rot_start, interleaved, eps):
    x = x.double().clone()
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    half = cos.shape[1]
    i = torch.arange(half, device=x.device)
    lo = rot_start + (2 * i if interleaved else i)
    hi = lo + (1 if interleaved else half)
    c, s = cos.double()[pos.long()][:, None], sin.double()[pos.long()][:, None]
    a, b = x[..., lo].clone(), x[..., hi].clone()
    x[..., lo], x[..., hi] = a * c - b * s, a * s + b * c
    return x


def norm_rope_close(got, ref, in_scale):
    # one bf16 rounding (ULP/2 of the value) and binary32 sums of 256 terms at most, whose errors are
    # relative to the terms of the rotation: 2^-18 of their size covers 64 roundings
    assert got.shape == ref.shape
    err = (got.double() - ref).abs()
    bound = ULP / 2 * 1.001 * ref.abs() + 2.0 ** -18 * in_scale
    assert bool((err <= bound).all()), float((err - bound).max())


@pytest.mark.parametrize("d,rot_start,rot,interleaved,norm", [
    (128, 0, 128, False, True),
    (128, 0, 128, True, True),
    (64, 0, 64, False, True),
    (64, 16, 32, True, False),
    (192, 128, 64, True, False),
    (192, 128, 64, False, True),
    (256, 0, 256, False, True),
    (16, 0, 16, False, True),
    (80, 8, 32, False, True),
    (240, 0, 0, False, True),
])
@pytest.mark.parametrize("T,hq,hk", [(1, 1, 1), (3, 7, 1), (17, 32, 8), (5, 3, 3)])
def test_norm_rope_without_cache(d, rot_start, rot, interleaved, norm, T, hq, hk):
    g = gen(d * 7 + T)
    q, k = rand(g, T, hq, d), rand(g, T, hk, d, scale=3.0)
    ang = torch.rand(50, rot // 2, generator=g, device="cuda") * 6.28
    cos, sin = ang.cos(), ang.sin()
    pos = torch.randint(0, 50, (T,), generator=g, device="cuda", dtype=torch.int32)
    qw = rand(g, d) if norm else None
    kw = rand(g, d) if norm else None
    qo, ko = fp8bs.qk_norm_rope(q, k, cos, sin, pos, q_weight=qw, k_weight=kw, eps=1e-5,
                                rot_start=rot_start, interleaved=interleaved)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        ref = norm_rope_ref(x, w, cos, sin, pos, rot_start, interleaved, 1e-5)
        norm_rope_close(got, ref, float(ref.abs().max()) * 1.5)


def test_norm_rope_one_weight_only():
    g = gen(3)
    q, k = rand(g, 4, 4, 128), rand(g, 4, 2, 128)
    cos, sin = torch.ones(8, 64, device="cuda"), torch.zeros(8, 64, device="cuda")
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    w = rand(g, 128)
    qo, ko = fp8bs.qk_norm_rope(q, k, cos, sin, pos, q_weight=w)
    norm_rope_close(qo, norm_rope_ref(q, w, cos, sin, pos, 0, False, 1e-6), 10.0)
    assert torch.equal(ko, k)          # neither norm nor turn: the same bits


@pytest.mark.parametrize("order", ["page-slot-head", "page-head-slot"])
@pytest.mark.parametrize("page,dk,dv", [(16, 128, 128), (1, 64, 64), (7, 192, 128), (64, 64, 128)])
def test_norm_rope_into_cache(order, page, dk, dv):
    g = gen(page)
    T, hq, hk, pages = 33, 6, 3, 60 // page + 3
    qkv = rand(g, T, hq * dk + hk * dk + hk * dv + 8)       # strided rows, padded
    q = qkv[:, :hq * dk].view(T, hq, dk)
    k = qkv[:, hq * dk:(hq + hk) * dk].view(T, hk, dk)
    v = qkv[:, (hq + hk) * dk:(hq + hk) * dk + hk * dv].view(T, hk, dv)
    cos, sin = (torch.rand(99, 32, generator=g, device="cuda") for _ in range(2))
    pos = torch.randint(0, 99, (T,), generator=g, device="cuda", dtype=torch.int32)
    w = rand(g, dk)
    if order == "page-slot-head":
        ck, cv = rand(g, pages, page, hk, dk), rand(g, pages, page, hk, dv)
    else:
        ck = rand(g, pages, hk, page, dk).transpose(1, 2)
        cv = rand(g, pages, hk, page, dv).transpose(1, 2)
    before_k, before_v = ck.clone(), cv.clone()
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].contiguous()
    slots[5] = -1                                           # padding: not written
    qo = fp8bs.qk_norm_rope(q, k, cos, sin, pos, q_weight=w, k_weight=w, rot_start=dk - 64,
                            cache=fp8bs.PagedCache(ck, cv), v=v, slots=slots)
    norm_rope_close(qo, norm_rope_ref(q, w, cos, sin, pos, dk - 64, False, 1e-6), 20.0)
    ref_k = norm_rope_ref(k, w, cos, sin, pos, dk - 64, False, 1e-6)
    for t in range(T):
        if t == 5:
            continue
        p, o = int(slots[t]) // page, int(slots[t]) % page
        norm_rope_close(ck[p, o], ref_k[t], 20.0)
        assert torch.equal(cv[p, o], v[t])
    touched = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
    touched[slots[slots >= 0]] = True
    touched = touched.view(pages, page)
    assert torch.equal(ck[~touched], before_k[~touched]) and torch.equal(cv[~touched], before_v[~touched])


def test_norm_rope_far_slots():
    # a cache whose slots lie past 2^32 bytes and 2^31 elements; only touched pages hold data
    pages, page, hk, d = 40000, 64, 8, 128
    ck = torch.empty(pages, page, hk, d, dtype=torch.bfloat16, device="cuda")
    cv = torch.empty(pages, page, hk, d, dtype=torch.bfloat16, device="cuda")
    g = gen(11)
    q, k, v = rand(g, 3, 8, d), rand(g, 3, hk, d), rand(g, 3, hk, d)
    cos, sin = (torch.rand(4, 64, generator=g, device="cuda") for _ in range(2))
    pos = torch.tensor([0, 3, 2], device="cuda", dtype=torch.int32)
    slots = torch.tensor([pages * page - 1, 2 ** 21 + 5, 0], device="cuda")
    fp8bs.qk_norm_rope(q, k, cos, sin, pos, cache=fp8bs.PagedCache(ck, cv), v=v, slots=slots)
    ref = norm_rope_ref(k, None, cos, sin, pos, 0, False, 1e-6)
    for t in range(3):
        norm_rope_close(ck.view(-1, hk, d)[slots[t]], ref[t], 10.0)
        assert torch.equal(cv.view(-1, hk, d)[slots[t]], v[t])


def test_norm_rope_reports_bad_indices():
    g = gen(12)
    q, k, v = rand(g, 3, 2, 64), rand(g, 3, 1, 64), rand(g, 3, 1, 64)
    cos, sin = (torch.rand(4, 32, generator=g, device="cuda") for _ in range(2))
    ck, cv = torch.zeros(2, 4, 1, 64, device="cuda").bfloat16(), torch.zeros(2, 4, 1, 64, device="cuda").bfloat16()
    pos = torch.tensor([1, 4, 2], device="cuda", dtype=torch.int32)
    slots = torch.tensor([8, 1, 2], device="cuda")
    qo = fp8bs.qk_norm_rope(q, k, cos, sin, pos, cache=fp8bs.PagedCache(ck, cv), v=v, slots=slots)
    assert fp8bs.fp8bs_device_error(clear=True) == fp8bs.DEVERR_INDEX
    assert bool((qo[1] == 0).all()) and bool((qo[0] != 0).any())
    assert torch.equal(cv.view(8, 1, 64)[2], v[2])
    cv.view(8, 1, 64)[2] = 0
    assert bool((cv == 0).all())


def test_norm_rope_empty():
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    t = torch.empty(5, 32, device="cuda")
    qo, ko = fp8bs.qk_norm_rope(e, e, t, t, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 4, 64)


# --------------------------------------------------------------------------- paged_attention

def paged_case(seed, news, lens, hq, hk, dk, dv, page, order="page-slot-head", spare=3, poison=True,
               q_scale=1.0):
    g = gen(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    if order == "page-slot-head":
        ck, cv = rand(g, pages, page, hk, dk), rand(g, pages, page, hk, dv)
    else:
        ck = rand(g, pages, hk, page, dk).transpose(1, 2)
        cv = rand(g, pages, hk, page, dv).transpose(1, 2)
    perm = torch.randperm(pages, generator=g, device="cuda").tolist()
    width = max(need + [1]) + 1
    table = torch.full((len(lens), width), -7, dtype=torch.int32)     # beyond the keys: never read
    used = torch.zeros(pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(need[b]):
            table[b, j] = perm.pop()
            used[table[b, j], :min(page, n - j * page)] = True
    if poison:          # whatever stands outside the keys must not be seen
        unused = ~used.cuda()
        ck[unused] = float("nan")
        cv[unused] = float("inf")
    T = sum(news)
    q = rand(g, T, hq, dk, scale=q_scale)
    starts = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32, device="cuda")
    return dict(q=q, cache=fp8bs.PagedCache(ck, cv), page_table=table.cuda(), q_start=starts,
                kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def attention_ref(c, news, lens, scale, causal, window):
    """(o, lse, sum of p |v|) in 64 bits."""
    q, (ck, cv) = c["q"], c["cache"]
    hq, hk = q.shape[1], ck.shape[2]
    page = ck.shape[1]
    o = torch.zeros(q.shape[0], hq, cv.shape[3], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(o)
    lse = torch.full((q.shape[0], hq), -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for b, (n, L) in enumerate(zip(news, lens)):
        j = torch.arange(L, device="cuda")
        pg = c["page_table"][b].long()[j // page]
        k = ck[pg, j % page].double().repeat_interleave(hq // hk, 1)
        v = cv[pg, j % page].double().repeat_interleave(hq // hk, 1)
        for i in range(n):
            hi = min(L, L - n + i + 1) if causal else L
            lo = max(0, L - n + i - window + 1) if window else 0
            if hi > lo:
                s = torch.einsum("hd,khd->hk", q[t + i].double(), k[lo:hi]) * scale
                lse[t + i] = torch.logsumexp(s, 1)
                p = torch.exp(s - lse[t + i][:, None])
                o[t + i] = torch.einsum("hk,khd->hd", p, v[lo:hi])
                mag[t + i] = torch.einsum("hk,khd->hd", p, v[lo:hi].abs())
        t += n
    return o, lse, mag


def attention_check(c, news, lens, scale=None, causal=True, window=0, **kw):
    dk = c["q"].shape[2]
    T, hq = c["q"].shape[:2]
    dv = c["cache"].v.shape[3]
    guard = torch.full((T + 2, hq, dv), 3.0, dtype=torch.bfloat16, device="cuda")
    out, lse = fp8bs.paged_attention(**c, scale=scale, causal=causal, window=window, return_lse=True,
                                     out=guard[1:T + 1], **kw)
    o, l, mag = attention_ref(c, news, lens, dk ** -0.5 if scale is None else scale, causal, window)
    assert bool((guard[0] == 3).all()) and bool((guard[T + 1] == 3).all())
    # probabilities rounded to bf16: ULP/2 of each term of sum p v; the output's rounding: ULP/2 of
    # |o| <= sum p |v|; binary32 scores (192 terms) and exponentials: 2^-12 of the sum covers them
    err = (out.double() - o).abs()
    bound = (ULP + 2.0 ** -12) * mag + 1e-30
    assert bool((err <= bound).all()), float((err / bound).max())
    empty = torch.isinf(l)
    assert bool((out[empty] == 0).all())
    assert torch.equal(torch.isinf(lse), empty) and bool((lse[empty] < 0).all())
    # lse: the scores' own error, 192 * 2^-24 * sum |q k| scale < 1e-4 for these inputs
    assert float((lse.double() - l)[~empty].abs().max() if bool((~empty).any()) else 0) <= 1e-4
    return out, lse


SHAPES = [(64, 64), (128, 128), (192, 128)]


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (8, 1), (7, 1), (6, 2), (32, 4)])
def test_attention_decode(dk, dv, hq, hk):
    lens = [1, 2, 63, 64, 65, 127, 128, 129, 300, 1000]
    news = [1] * len(lens)
    attention_check(paged_case(1, news, lens, hq, hk, dk, dv, 16), news, lens)


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("news,lens", [
    ([128], [128]), ([1], [1]), ([129], [129]), ([200], [333]), ([64, 1, 0, 17], [64, 500, 30, 17]),
    ([300, 5], [300, 1029]), ([2, 2, 2], [2, 130, 257]),
])
@pytest.mark.parametrize("hq,hk", [(4, 4), (4, 1), (6, 2)])
def test_attention_chunks(dk, dv, news, lens, hq, hk):
    attention_check(paged_case(2, news, lens, hq, hk, dk, dv, 32), news, lens)


@pytest.mark.parametrize("page", [1, 5, 16, 48, 64, 128, 200, 256])
@pytest.mark.parametrize("order", ["page-slot-head", "page-head-slot"])
def test_attention_page_sizes(page, order):
    news, lens = [1, 40, 3], [517, 200, 3]
    attention_check(paged_case(3, news, lens, 8, 2, 128, 128, page, order), news, lens)


@pytest.mark.parametrize("window", [1, 2, 100, 128, 5000])
@pytest.mark.parametrize("hq,hk", [(4, 4), (8, 1)])
def test_attention_window(window, hq, hk):
    news, lens = [1, 150, 1, 0, 20], [1000, 400, 1, 9, 777]
    attention_check(paged_case(4, news, lens, hq, hk, 64, 64, 16), news, lens, window=window)


@pytest.mark.parametrize("page", [1, 5, 16, 64, 128])
@pytest.mark.parametrize("T", [1, 20, 200])
def test_attention_window_over_freed_pages(page, T):
    # pages that end before the window have been given back: their entries are out of the cache, and their
    # contents not numbers
    news, lens, window = [T, 1], [1500, 700], 150
    c = paged_case(16, news, lens, 4, 2, 128, 128, page)
    ref = fp8bs.paged_attention(**c, window=window, return_lse=True)
    for b, (n, L) in enumerate(zip(news, lens)):
        gone = max(0, L - n - window + 1) // page
        c["cache"].k[c["page_table"][b, :gone].long()] = float("nan")
        c["cache"].v[c["page_table"][b, :gone].long()] = float("inf")
        c["page_table"][b, :gone] = -1
    out = fp8bs.paged_attention(**c, window=window, return_lse=True)
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    assert bool(torch.isfinite(out[0].float()).all())


def test_attention_reports_bad_lengths():
    # one sequence past the caller's bounds: reported, and the others as ever
    news, lens = [1, 1, 3], [100, 60, 40]
    c = paged_case(17, news, lens, 4, 2, 64, 64, 16)
    ref = fp8bs.paged_attention(**c)
    c["kv_len"][1] = 10 ** 6
    out = fp8bs.paged_attention(**c)
    assert fp8bs.fp8bs_device_error(clear=True) == fp8bs.DEVERR_INDEX
    assert torch.equal(out[0], ref[0]) and torch.equal(out[2:], ref[2:])


@pytest.mark.parametrize("B", [257, 700])
def test_attention_many_sequences(B):
    # more sequences than one look-up chunk holds, of every length, some without queries
    news = [(b * 7) % 4 for b in range(B)]
    lens = [max(n, (b * 13) % 90) for b, n in enumerate(news)]
    attention_check(paged_case(18, news, lens, 2, 1, 64, 64, 16), news, lens)


def test_scratch_memory_of_a_captured_graph_outlives_larger_calls():
    news, lens = [1], [3000]
    small = paged_case(19, news, lens, 8, 2, 128, 128, 16)
    large = paged_case(20, [1] * 200, [3000] * 200, 8, 2, 128, 128, 16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ref = fp8bs.paged_attention(**small)
        out = torch.empty_like(ref)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            fp8bs.paged_attention(**small, out=out)
        big = fp8bs.paged_attention(**large)
        other = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(40)]
        s.synchronize()
        out.zero_()
        graph.replay()
        s.synchronize()
    assert torch.equal(out, ref) and bool(torch.isfinite(big.float()).all())
    assert all(bool((o == 7).all()) for o in other)


@pytest.mark.parametrize("window", [0, 50])
def test_attention_not_causal(window):
    news, lens = [7, 130, 1], [300, 130, 0]
    attention_check(paged_case(5, news, lens, 4, 2, 128, 128, 16), news, lens, causal=False,
                    window=window)


def test_attention_rows_without_keys():
    # more new tokens than keys: the first ones see nothing; and a sequence without any key
    news, lens = [10, 3, 200], [4, 0, 60]
    out, lse = attention_check(paged_case(6, news, lens, 4, 2, 128, 128, 16), news, lens)
    assert bool(torch.isinf(lse[:6]).all()) and bool(torch.isinf(lse[10:13]).all())


@pytest.mark.parametrize("T,L,hq,hk", [(1, 20000, 8, 1), (1, 9999, 2, 2), (4, 12345, 8, 2)])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_attention_long_keys(T, L, hq, hk, dk, dv):
    attention_check(paged_case(7, [T], [L], hq, hk, dk, dv, 64), [T], [L])


def test_attention_long_chunk():
    attention_check(paged_case(8, [700], [1700], 8, 2, 128, 128, 64), [700], [1700])


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("n,L,hq,hk,window,causal", [
    (1999, 2300, 24, 8, 0, True),      # 192 tiles of rows: one whole round of CTAs and a part of one
    (2500, 2500, 32, 8, 0, True),      # 320: two and a part
    (1230, 3001, 32, 16, 500, True),   # 160, a window
    (1230, 1300, 16, 8, 0, False),     # 80: less than a round
])
def test_attention_rounds_of_one_sequence(dk, dv, n, L, hq, hk, window, causal):
    attention_check(paged_case(17, [n], [L], hq, hk, dk, dv, 32), [n], [L], window=window, causal=causal)


def test_attention_rounds_of_a_batch():
    news, lens = [700, 1, 1100, 300], [700, 900, 1500, 2001]
    attention_check(paged_case(18, news, lens, 32, 16, 128, 128, 16), news, lens)


@pytest.mark.parametrize("scale", [0.0, 1.0, 3.0])
def test_attention_scales(scale):
    # flat, and almost one key only: large scores, whose maximum moves a lot between tiles. Scores grow
    # with the scale, and their binary32 error with them: 1e-4 holds to |s| ~ 60 (192 * 2^-24 * 5 * 60
    # is 3e-3 in the worst case, its root mean square 1e-4 / 4)
    news, lens = [1, 130], [600, 700]
    attention_check(paged_case(9, news, lens, 4, 2, 64, 64, 16), news, lens, scale=scale)


def test_attention_strided_queries_and_tight_bounds():
    news, lens = [5, 1], [90, 333]
    c = paged_case(10, news, lens, 4, 2, 128, 128, 16)
    wide = torch.zeros(6, 9, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:7] = c["q"]
    c["q"] = wide[:, 3:7]
    attention_check(c, news, lens, max_q_len=5, max_kv_len=333)


def test_attention_same_bits_twice_and_on_another_stream():
    news, lens = [1, 1, 30], [5000, 77, 800]
    c = paged_case(11, news, lens, 8, 2, 128, 128, 16)
    a = fp8bs.paged_attention(**c, return_lse=True)
    b = fp8bs.paged_attention(**c, return_lse=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        d = fp8bs.paged_attention(**c, return_lse=True)
    s.synchronize()
    for x, y, z in zip(a, b, d):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_attention_far_pages():
    # pages past 2^31 elements and 2^32 bytes of the cache
    pages, page, hk, d = 40000, 64, 8, 128
    ck = torch.empty(pages, page, hk, d, dtype=torch.bfloat16, device="cuda")
    cv = torch.empty(pages, page, hk, d, dtype=torch.bfloat16, device="cuda")
    g = gen(13)
    ids = [39999, 17, 33333, 32769]
    for i in ids:
        ck[i], cv[i] = rand(g, page, hk, d), rand(g, page, hk, d)
    c = dict(q=rand(g, 2, 16, d), cache=fp8bs.PagedCache(ck, cv),
             page_table=torch.tensor([ids], dtype=torch.int32, device="cuda"),
             q_start=torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
             kv_len=torch.tensor([250], dtype=torch.int32, device="cuda"))
    attention_check(c, [2], [250])


def test_attention_reports_bad_pages():
    news, lens = [1], [100]
    c = paged_case(14, news, lens, 2, 1, 64, 64, 16, poison=False)
    c["page_table"][0, 2] = 10 ** 6
    out = fp8bs.paged_attention(**c)
    assert fp8bs.fp8bs_device_error(clear=True) == fp8bs.DEVERR_INDEX
    assert bool(torch.isfinite(out.float()).all())


def test_attention_graph_replay():
    news, lens = [1, 1], [3000, 200]
    c = paged_case(15, news, lens, 8, 2, 128, 128, 16)
    ref = fp8bs.paged_attention(**c)
    torch.cuda.synchronize()
    out = torch.empty_like(ref)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        fp8bs.paged_attention(**c, out=out)     # the stream's workspace is made before the capture
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            fp8bs.paged_attention(**c, out=out)
    out.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


# ---------------------------------------------------------------------------------- moe layer

def quant_ref(x, ue8m0):
    """Block quantisation of binary32 values: (values the codes stand for) in binary64."""
    b = x.float().double().unflatten(-1, (-1, 128))
    s = (b.abs().amax(-1, keepdim=True).clamp(min=float(np.float32(1e-4))) / 448.0).float().double()
    if ue8m0:
        m, e = torch.frexp(s)
        s = ((torch.where(m > 0.5, e, e - 1).long() + 1023) << 52).view(torch.float64)
    v = (b / s).float().double()
    _, e = torch.frexp(v)
    ulp = (((e - 4).clamp(min=-9).long() + 1023) << 52).view(torch.float64)
    return ((torch.round(v / ulp) * ulp).clamp(-448, 448) * s).flatten(-2)


def moe_weights(g, E, rows, cols, pow2=False):
    codes = (torch.randn(E, rows, cols, generator=g, device="cuda") * 32).to(torch.float8_e4m3fn)
    s = torch.exp2(torch.rand(E, rows // 128, cols // 128, generator=g, device="cuda") * 2 - 1)
    s = s / (32 * math.sqrt(cols))
    return codes, torch.exp2(torch.round(torch.log2(s))) if pow2 else s


def moe_ref(x, weights, ids, w13, s13, w2, s2, ue8m0):
    """(y, tolerance) in 64 bits. The tolerance: one bf16 rounding of y; for each of a token's experts
    one code of h on the other side of a rounding boundary (the binary32 sums before it are not the
    64-bit ones), which moves one term by at most its eighth; and 2^-18 of all terms for binary32 sums."""
    inter = w2.shape[2]
    y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    flip, size = torch.zeros_like(y), torch.zeros_like(y)
    xq = quant_ref(x, ue8m0)

    def deq(c, s):
        return c.double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)

    for e in range(w2.shape[0]):
        rows, slot = torch.where(ids == e)
        if not len(rows):
            continue
        gu = xq[rows] @ deq(w13[e], s13[e]).T
        h = quant_ref(gu[:, :inter] * torch.sigmoid(gu[:, :inter]) * gu[:, inter:], ue8m0)
        W = deq(w2[e], s2[e])
        w = weights[rows, slot].double()[:, None]
        y.index_add_(0, rows, w * (h @ W.T))
        size.index_add_(0, rows, w.abs() * (h.abs() @ W.abs().T))
        big = torch.stack([(r.abs()[None] * W.abs()).amax(1) for r in h])
        flip.index_add_(0, rows, w.abs() * big / 8)
    return y, ULP / 2 * 1.001 * y.abs() + flip + 2.0 ** -18 * size


def moe_close(got, ref):
    y, tol = ref
    err = (got.double() - y).abs()
    assert bool((err <= tol + 1e-30).all()), float((err / tol).max())


@pytest.mark.parametrize("T,D,I,E,k", [
    (1, 128, 128, 1, 1), (1, 256, 128, 8, 2), (2, 512, 256, 16, 4), (5, 384, 640, 8, 3),
    (16, 256, 256, 4, 2), (17, 256, 128, 64, 8), (33, 640, 256, 8, 2), (64, 256, 384, 32, 8),
    (64, 1024, 128, 3, 3), (3, 128, 256, 300, 32), (7, 7168, 256, 8, 2), (2, 256, 2048, 8, 8),
    (48, 2048, 512, 16, 6),
])
@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
def test_moe_experts(T, D, I, E, k, fmt):
    g = gen(T * 31 + D + I)
    x = rand(g, T, D)
    w13, s13 = moe_weights(g, E, 2 * I, D, fmt == "ue8m0")
    w2, s2 = moe_weights(g, E, D, I, fmt == "ue8m0")
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    weights = torch.rand(T, k, generator=g, device="cuda")
    guard = torch.full((T + 2, D), 3.0, dtype=torch.bfloat16, device="cuda")
    y = fp8bs.moe_experts(x, weights, ids, w13, s13, w2, s2, scale_fmt=fmt, out=guard[1:T + 1])
    moe_close(y, moe_ref(x, weights, ids, w13, s13, w2, s2, fmt == "ue8m0"))
    assert bool((guard[0] == 3).all()) and bool((guard[T + 1] == 3).all())
    again = fp8bs.moe_experts(x, weights, ids, w13, s13, w2, s2, scale_fmt=fmt)
    assert torch.equal(y, again)


@pytest.mark.parametrize("T,D,I,E,k", [
    (1, 1024, 128, 4, 1), (3, 4480, 512, 8, 1), (5, 4736, 128, 24, 4), (20, 1536, 128, 8, 2), (64, 2176, 128, 4, 2),
    (64, 4096, 256, 2, 2),
])
@pytest.mark.parametrize("same", [False, True])
def test_moe_few_items_for_the_gpu(T, D, I, E, k, same):
    # `same`: all tokens choose the same experts, so that fewer are met than there could be
    g = gen(T + D + I)
    x = rand(g, T, D)
    w13, s13 = moe_weights(g, E, 2 * I, D, False)
    w2, s2 = moe_weights(g, E, D, I, False)
    ids = torch.stack([torch.arange(k, device="cuda") if same else
                       torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    weights = torch.rand(T, k, generator=g, device="cuda")
    y = fp8bs.moe_experts(x, weights, ids, w13, s13, w2, s2)
    moe_close(y, moe_ref(x, weights, ids, w13, s13, w2, s2, False))
    assert torch.equal(y, fp8bs.moe_experts(x, weights, ids, w13, s13, w2, s2))


def test_moe_experts_absent_repeated_and_bad_ids():
    g = gen(5)
    T, D, I, E, k = 6, 256, 256, 4, 3
    x = rand(g, T, D)
    w13, s13 = moe_weights(g, E, 2 * I, D)
    w2, s2 = moe_weights(g, E, D, I)
    ids = torch.tensor([[0, 1, -1], [-1, -1, -1], [2, 2, 3], [3, 0, 1], [1, 1, 1], [-1, 2, -1]],
                       dtype=torch.int32, device="cuda")
    weights = torch.randn(T, k, generator=g, device="cuda")
    ref = moe_ref(x, weights, ids, w13, s13, w2, s2, False)
    y = fp8bs.moe_experts(x, weights, ids, w13, s13, w2, s2)
    moe_close(y, ref)
    assert bool((y[1] == 0).all())
    bad = torch.where(ids < 0, torch.tensor(4, device="cuda", dtype=torch.int32), ids)
    y2 = fp8bs.moe_experts(x, weights, bad, w13, s13, w2, s2)
    assert fp8bs.fp8bs_device_error(clear=True) == fp8bs.DEVERR_INDEX
    assert torch.equal(y, y2)
    none = fp8bs.moe_experts(x, weights, torch.full_like(ids, -1), w13, s13, w2, s2)
    assert bool((none == 0).all())


def test_moe_one_token_does_not_disturb_another():
    # a token of infinities and one of zeros beside ordinary ones
    g = gen(6)
    T, D, I, E, k = 5, 256, 256, 8, 2
    x = rand(g, T, D)
    w13, s13 = moe_weights(g, E, 2 * I, D)
    w2, s2 = moe_weights(g, E, D, I)
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    weights = torch.rand(T, k, generator=g, device="cuda")
    plain = fp8bs.moe_experts(x, weights, ids, w13, s13, w2, s2)
    x2 = x.clone()
    x2[1] = float("inf")
    x2[3] = 0
    y = fp8bs.moe_experts(x2, weights, ids, w13, s13, w2, s2)
    for t in (0, 2, 4):
        assert torch.equal(y[t], plain[t])
    assert bool((y[3] == 0).all())


def test_moe_empty():
    g = gen(7)
    w13, s13 = moe_weights(g, 2, 256, 128)
    w2, s2 = moe_weights(g, 2, 128, 128)
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    y = fp8bs.moe_layer(e, rand(g, 2, 128), w13, s13, w2, s2, top_k=1)
    assert y.shape == (0, 128)


def route_ref(logits, k, bias, score, groups, topk_groups, normalise, scale):
    """In 64 bits, one token at a time; ties to the lowest index."""
    weights, ids = [], []
    for row in logits.double().cpu().numpy():
        s = 1 / (1 + np.exp(-row)) if score == "sigmoid" else np.exp(row - row.max()) / np.exp(row - row.max()).sum()
        c = s + (0 if bias is None else bias.double().cpu().numpy())
        by = c.reshape(groups, -1)
        top = np.sort(by, 1)[:, ::-1]
        rank = top[:, 0] if bias is None else top[:, :2].sum(1)
        keep = np.argsort(-rank, kind="stable")[:topk_groups]
        shut = np.full_like(by, -np.inf)
        shut[keep] = by[keep]
        i = np.argsort(-shut.ravel(), kind="stable")[:k]
        w = s[i] / (s[i].sum() if normalise else 1) * scale
        weights.append(w)
        ids.append(i)
    return np.stack(weights), np.stack(ids)


@pytest.mark.parametrize("E,k,groups,topk_groups", [
    (1, 1, 1, 1), (8, 2, 1, 1), (32, 8, 8, 4), (256, 8, 8, 4), (512, 32, 32, 8), (24, 6, 3, 2),
    (33, 5, 1, 1),
])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
def test_moe_route(E, k, groups, topk_groups, score, biased):
    # x picks single channels, so the logits are the router's bf16 weights themselves: multiples of
    # 1/64, many of them equal (ties), the others further apart than any rounding
    T, D = 37, 128
    g = gen(E + k)
    router = (torch.randint(-128, 128, (E, D), generator=g, device="cuda") / 64).bfloat16()
    x = torch.zeros(T, D, device="cuda")
    x[torch.arange(T), torch.randperm(D, generator=g, device="cuda")[:T]] = 1
    x = x.bfloat16()
    bias = torch.randint(0, 3, (E,), generator=g, device="cuda").float() * 4 if biased else None
    w, ids = fp8bs.moe_route(x, router, k, bias=bias, score=score, groups=groups,
                             topk_groups=topk_groups, route_scale=2.5)
    rw, rid = route_ref(x.double() @ router.double().T, k, bias, score, groups, topk_groups,
                        score == "sigmoid", 2.5)
    assert np.array_equal(ids.cpu().numpy(), rid)
    # binary32: a sum over 512 experts and a few roundings
    assert np.all(np.abs(w.double().cpu().numpy() - rw) <= 2.0 ** -19 * rw)


@pytest.mark.parametrize("T,D,E", [(1, 7168, 32), (9, 2048, 64), (200, 640, 16), (5, 16384, 8)])
def test_moe_route_sums(T, D, E):
    # all experts chosen: the weights of each expert against 64-bit sums
    g = gen(D)
    x, router = rand(g, T, D), rand(g, E, D, scale=D ** -0.5)
    k = min(E, 32)
    w, ids = fp8bs.moe_route(x, router, k, normalise=False)
    logits = x.double() @ router.double().T
    ref = torch.sigmoid(torch.take_along_dim(logits, ids.long(), 1))
    assert int(ids.min()) >= 0 and int(ids.max()) < E
    assert bool((ids.sort(1)[0].diff(dim=1) > 0).all())
    # lanes add up to 16384 / 256 terms in a row, then 13 levels: 80 roundings of sums of size ~3
    assert float((w.double() - ref).abs().max()) <= 80 * 2.0 ** -24 * 3


def test_moe_layer_is_route_then_experts():
    g = gen(21)
    T, D, I, E = 11, 512, 256, 16
    x, router = rand(g, T, D), rand(g, E, D, scale=0.05)
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    w13, s13 = moe_weights(g, E, 2 * I, D)
    w2, s2 = moe_weights(g, E, D, I)
    w, ids = fp8bs.moe_route(x, router, 4, bias=bias, groups=4, topk_groups=2)
    y = fp8bs.moe_experts(x, w, ids, w13, s13, w2, s2)
    z = fp8bs.moe_layer(x, router, w13, s13, w2, s2, 4, bias=bias, groups=4, topk_groups=2)
    assert torch.equal(y, z)


def test_moe_layer_graph_replay():
    g = gen(22)
    T, D, I, E = 3, 512, 256, 16
    x, router = rand(g, T, D), rand(g, E, D, scale=0.05)
    w13, s13 = moe_weights(g, E, 2 * I, D)
    w2, s2 = moe_weights(g, E, D, I)
    y = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fp8bs.moe_layer(x, router, w13, s13, w2, s2, 4, out=y)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            fp8bs.moe_layer(x, router, w13, s13, w2, s2, 4, out=y)
    torch.cuda.synchronize()
    x.copy_(rand(g, T, D))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, fp8bs.moe_layer(x, router, w13, s13, w2, s2, 4))
