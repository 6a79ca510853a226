"""The operators around the FP8 products of a decoder layer at the edges of what they accept."""
import threading

import pytest
import torch

import fp8_block_scaled_fp8bs_gb300 as fp8bs
from test_layer_gpu import (attention_check, gen, moe_close, moe_ref, moe_weights, no_device_error,  # noqa: F401
                            norm_rope_close, norm_rope_ref, paged_case, rand)

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


# --------------------------------------------------------------------------- scores that are not finite

def not_finite_case(dk, dv, n, L):
    c = paged_case(61, [n], [L], 8, 2, dk, dv, 16)
    q, k = c["q"], c["cache"].k

    def key(j, head):
        return k[int(c["page_table"][0, j // 16]), j % 16, head]

    pages = c["page_table"][0, :-(-L // 16)].long()
    k[pages, :, 1, 9] = k[pages, :, 1, 9].abs() + 0.125
    q[0, 0] = float("nan")                                   # a query: all its scores are NaN
    q[0, 1, 5] = float("inf")                                # scores of both infinities, then
    key(2, 1)[7] = float("inf")                              # one key: +-infinity by the query's sign
    key(L - 1, 0)[3] = float("nan")                          # one key of the last query alone
    q[0, 6] = 0
    q[0, 6, 9], q[0, 6, 7] = -float("inf"), -1               # all scores -infinity
    return c


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("n,L", [(1, 40), (1, 20000), (5, 3000), (300, 400), (300, 6000)])
def test_scores_that_are_not_finite(dk, dv, n, L):
    # one tile of queries and two, in one piece of the keys and in many
    c = not_finite_case(dk, dv, n, L)
    out, lse = fp8bs.paged_attention(**c, return_lse=True)
    j = torch.arange(L, device="cuda")
    pg = c["page_table"][0].long()[j // 16]
    k = c["cache"].k[pg, j % 16].double().repeat_interleave(4, 1)
    v = c["cache"].v[pg, j % 16].double().repeat_interleave(4, 1)
    s = torch.einsum("nhd,khd->nhk", c["q"].double(), k) * dk ** -0.5
    s[0, 6] = -float("inf")                 # (in the sum above its zeros meet the infinity of one key's channel)
    seen = (j <= L - n + torch.arange(n, device="cuda")[:, None])[:, None]
    bad = ((torch.isnan(s) | (s == float("inf"))) & seen).any(-1)
    s = s.masked_fill(~seen, -float("inf"))
    none = ~bad & torch.isinf(s).all(-1)
    assert bool(bad[0, :2].all()) and bool(none[0, 6]) and int(none.sum()) == 1 and not bool(bad[:, 4:].all())
    assert bool(torch.isnan(out[bad].float()).all()) and bool(torch.isnan(lse[bad]).all())
    assert bool((out[none] == 0).all()) and bool((lse[none] == -float("inf")).all())
    good = ~bad & ~none
    l = torch.logsumexp(s, -1)
    p = torch.exp(s - l[..., None])
    p[~good] = 0
    o = torch.einsum("nhk,khd->nhd", p, v)
    mag = torch.einsum("nhk,khd->nhd", p, v.abs())
    # as in attention_check: probabilities and output rounded to bf16, binary32 scores and sums
    err = (out.double() - o).abs()
    assert bool((err <= (2.0 ** -7 + 2.0 ** -12) * mag + 1e-30)[good].all())
    assert bool(((lse.double() - l)[good].abs() <= 1e-4).all())


@pytest.mark.parametrize("n,L", [(1, 40), (1, 20000), (300, 400)])
def test_a_scale_that_is_not_a_number(n, L):
    c = paged_case(62, [n], [L], 8, 2, 128, 128, 16)
    out, lse = fp8bs.paged_attention(**c, scale=float("nan"), return_lse=True)
    assert bool(torch.isnan(out.float()).all()) and bool(torch.isnan(lse).all())


# ------------------------------------------------------------------------- bounds far above the lengths

@pytest.mark.parametrize("B,n,hq,hk,dk,dv,kv", [
    (150, 16, 64, 8, 128, 128, 131072),       # a page table for long conversations, short chunks
    (64, 1, 64, 8, 128, 128, 1 << 20),
    (1, 1, 32, 8, 128, 128, 1 << 30),
    (128, 1, 128, 8, 192, 128, 65536),
    (64, 1, 16, 16, 64, 64, 1 << 24),
    (1, 8192, 64, 1, 128, 128, 1 << 20),      # one chunk: two query tiles
    (4, 1, 16, 4, 128, 128, 33000),
])
def test_workspace_is_bounded(B, n, hq, hk, dk, dv, kv):
    torch.cuda.init()
    a = fp8bs.PagedAttentionArgs(
        cache=fp8bs.KvCache(pages=1, page_size=16, heads=hk, dk=dk, dv=dv), table_stride=-(-kv // 16), B=B, T=B * n,
        q_heads=hq, max_q_len=n, max_kv_len=kv, causal=1, scale=1.0)
    assert fp8bs.fp8bs_paged_attention_workspace_size(a) <= 1 << 29


@pytest.mark.parametrize("news,lens", [([1] * 30, [10 * b + 1 for b in range(30)]), ([16] * 30, [300] * 30),
                                       ([500, 1], [500, 3000])])
def test_tables_far_wider_than_the_sequences(news, lens):
    c = paged_case(71, news, lens, 64, 8, 64, 64, 16)
    wide = torch.full((len(lens), 1 << 20), -7, dtype=torch.int32, device="cuda")
    wide[:, :c["page_table"].shape[1]] = c["page_table"]
    c["page_table"] = wide
    attention_check(c, news, lens)


# -------------------------------------------------------------------------------- several host threads

def test_host_threads_with_layers_of_different_sizes():
    # what one thread's calls set for a kernel must suit the other's: the shared memory of both kernels depends
    # on the sizes. (The raw calls: they let other threads run.)
    g = gen(81)
    fp8bs.load()

    def case(D, E, I, T):
        x, router = rand(g, T, D), rand(g, E, D, scale=0.02)
        w13, s13 = moe_weights(g, 2, 2 * I, D)
        w2, s2 = moe_weights(g, 2, D, I)
        ids = torch.randint(0, 2, (T, 1), generator=g, device="cuda", dtype=torch.int32)
        one = torch.ones(T, 1, device="cuda")
        routing = fp8bs.MoeRouting(router_w=router.data_ptr(), top_k=2, groups=1, topk_groups=1, score=0, normalise=1,
                                   route_scale=1.0)
        size = fp8bs.fp8bs_moe_workspace_size(T, D, I, 2, 1)
        work = torch.empty(size, dtype=torch.uint8, device="cuda")
        weights = torch.empty(T, 2, device="cuda")
        chosen = torch.empty(T, 2, dtype=torch.int32, device="cuda")
        y = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")

        def call(stream):
            fp8bs.fp8bs_moe_route(x.data_ptr(), routing, weights.data_ptr(), chosen.data_ptr(), T, D, E, stream)
            fp8bs.fp8bs_moe_experts(x.data_ptr(), one.data_ptr(), ids.data_ptr(), w13.data_ptr(), s13.data_ptr(),
                                    w2.data_ptr(), s2.data_ptr(), y.data_ptr(), T, D, I, 2, 1, workspace=work.data_ptr(),
                                    workspace_bytes=size, stream=stream)
        keep = (x, router, w13, s13, w2, s2, ids, one, work, routing)
        return call, lambda: (weights.clone(), chosen.clone(), y.clone()), keep

    cases = [case(16384, 512, 128, 3), case(128, 8, 128, 3)]
    refs = []
    for call, results, _ in cases:
        call(0)
        torch.cuda.synchronize()
        refs.append(results())
    failed = []

    def run(call):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            for i in range(2000):
                call(stream.cuda_stream)
                if i % 100 == 99:
                    stream.synchronize()
            stream.synchronize()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=run, args=(call,)) for call, _, _ in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for (_, results, _), ref in zip(cases, refs):
        assert all(torch.equal(a, b) for a, b in zip(results(), ref))


# ------------------------------------------------------------------------- far ends of what is accepted

@pytest.mark.parametrize("d,rot_start,rot,interleaved", [(64, 0, 64, False), (64, 16, 32, True), (128, 0, 128, True),
                                                         (128, 0, 128, False), (192, 128, 64, True), (256, 0, 256, False)])
@pytest.mark.parametrize("T,hq,hk", [(2048, 7, 3), (2500, 1, 1), (5001, 3, 2)])
def test_norm_rope_of_many_tokens(d, rot_start, rot, interleaved, T, hq, hk):
    # the form for long chunks, with rows of q, k and v beside one another and a cache of odd pages
    g = gen(T + d)
    qkv = rand(g, T, (hq + 2 * hk) * d)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hk * d, hk * d], 1))
    pages = T // 7 + 2
    ck, cv = rand(g, pages, 7, hk, d), rand(g, pages, 7, hk, d)
    before_k, before_v = ck.clone(), cv.clone()
    ang = torch.rand(99, rot // 2, generator=g, device="cuda") * 6.28
    pos = torch.randint(0, 99, (T,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(pages * 7, generator=g, device="cuda")[:T].contiguous()
    slots[T // 2] = -1
    w = rand(g, d)
    qo = fp8bs.qk_norm_rope(q, k, ang.cos(), ang.sin(), pos, q_weight=w, k_weight=w, rot_start=rot_start,
                            interleaved=interleaved, cache=fp8bs.PagedCache(ck, cv), v=v, slots=slots)
    ref = norm_rope_ref(q, w, ang.cos(), ang.sin(), pos, rot_start, interleaved, 1e-6)
    norm_rope_close(qo, ref, float(ref.abs().max()) * 1.5)
    ref = norm_rope_ref(k, w, ang.cos(), ang.sin(), pos, rot_start, interleaved, 1e-6)
    there = slots >= 0
    norm_rope_close(ck.view(-1, hk, d)[slots[there]], ref[there], float(ref.abs().max()) * 1.5)
    assert torch.equal(cv.view(-1, hk, d)[slots[there]], v[there])
    rest = torch.ones(pages * 7, dtype=torch.bool, device="cuda")
    rest[slots[there]] = False
    rest = rest.view(pages, 7)
    assert torch.equal(ck[rest], before_k[rest]) and torch.equal(cv[rest], before_v[rest])


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("hq,hk", [(20, 1), (128, 1), (130, 1), (600, 2)])
@pytest.mark.parametrize("news,lens", [([1, 1], [700, 33]), ([1], [9000]), ([5, 1, 3], [5, 300, 1000])])
def test_attention_of_many_query_heads_to_a_key_head(dk, dv, hq, hk, news, lens):
    attention_check(paged_case(91, news, lens, hq, hk, dk, dv, 16), news, lens)


@pytest.mark.parametrize("dk,dv", [(64, 64), (192, 128)])
@pytest.mark.parametrize("news,lens", [([1, 1], [700, 12000]), ([150, 1], [150, 300])])
def test_attention_negative_scale(dk, dv, news, lens):
    attention_check(paged_case(92, news, lens, 8, 2, dk, dv, 16), news, lens, scale=-0.125)


@pytest.mark.parametrize("T,D,I,E,k", [
    (1, 16384, 128, 4, 2), (5, 16384, 256, 4, 2), (20, 16384, 128, 4, 2), (64, 16384, 256, 3, 2),
    (1, 128, 16384, 3, 1), (9, 256, 16384, 3, 2), (64, 128, 16384, 2, 2),
    (2, 512, 256, 16, 4), (7, 2048, 1024, 8, 2), (33, 1024, 512, 12, 3), (64, 512, 1024, 16, 8),
])
@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
def test_moe_experts_as_a_whole(T, D, I, E, k, fmt):
    # Beside the bound of each output, which allows each a code on the other side of a rounding boundary, the size of all
    # errors together. y's rounding to bf16 is at most 2^-8 of its size. A code goes the other way where h is within its
    # binary32 error (2^-16 of it, say) of a boundary; these are 2^-4 of it apart, so one code in 2^11 does, and moves its
    # term by 2^-3 at most: 2^-3 / sqrt(2^11) < 2^-8 of the size. A lost block of 128 of the k * I terms would be
    # sqrt(128 / (k I)), 2^-4 or more here.
    g = gen(T * 17 + D + I)
    x = rand(g, T, D)
    w13, s13 = moe_weights(g, E, 2 * I, D, fmt == "ue8m0")
    w2, s2 = moe_weights(g, E, D, I, fmt == "ue8m0")
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    weights = torch.rand(T, k, generator=g, device="cuda") + 0.5
    y = fp8bs.moe_experts(x, weights, ids, w13, s13, w2, s2, scale_fmt=fmt)
    ref = moe_ref(x, weights, ids, w13, s13, w2, s2, fmt == "ue8m0")
    moe_close(y, ref)
    assert float((y.double() - ref[0]).norm() / ref[0].norm()) <= 2.0 ** -7
