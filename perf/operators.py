"""Cases of the operators around the FP8 products of a decoder layer, for measurement:

  qk_norm_rope      norms of queries and keys per head, position rotation, write into the cache
  paged_attention   attention of a chunk of new tokens over a paged cache
  moe_layer         router, experts and weighted sum of a mixture-of-experts layer, few tokens

`run` computes each in its plain form (elementary torch operations in 32 bits) or, with `own`,
through the package's entry points; `exact` computes it from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128


def listed():
    return [
        # a decode step of five sequences (odd): query/key norms, rotation in halves
        {"name": "norm_rope_decode5", "op": "norm_rope", "tokens": 5, "q_heads": 32,
         "k_heads": 8, "dk": 128, "dv": 128, "rot": 128, "rot_start": 0, "interleaved": False,
         "norm": True, "page": 64},
        # a long prefill chunk of the same layer
        {"name": "norm_rope_chunk8192", "op": "norm_rope", "tokens": 8192, "q_heads": 32,
         "k_heads": 8, "dk": 128, "dv": 128, "rot": 128, "rot_start": 0, "interleaved": False,
         "norm": True, "page": 64},
        # latent-attention heads expanded to 128 + 64 channels: only the last 64 rotate, no norm
        {"name": "norm_rope_mla1000", "op": "norm_rope", "tokens": 1000, "q_heads": 16,
         "k_heads": 16, "dk": 192, "dv": 128, "rot": 64, "rot_start": 128, "interleaved": True,
         "norm": False, "page": 64},
        # one token of one long conversation: latency and the split over the key axis
        {"name": "attn_decode1_32k", "op": "attention", "new": 1, "seqs": 1, "kv": 32785,
         "ragged": False, "q_heads": 32, "k_heads": 8, "dk": 128, "dv": 128, "page": 64,
         "window": 0},
        # a decode batch of conversations of all lengths
        {"name": "attn_decode64_ragged", "op": "attention", "new": 1, "seqs": 64, "kv": 8192,
         "ragged": True, "q_heads": 64, "k_heads": 8, "dk": 128, "dv": 128, "page": 16,
         "window": 0},
        # the second half of a long prompt, prefilled as one chunk over the cached first half
        {"name": "attn_chunk4096", "op": "attention", "new": 4096, "seqs": 1, "kv": 8192,
         "ragged": False, "q_heads": 32, "k_heads": 8, "dk": 128, "dv": 128, "page": 64,
         "window": 0},
        # chunks and decodes mixed in one batch, sliding window, as many key heads as query heads
        {"name": "attn_mixed8_window", "op": "attention", "new": 300, "seqs": 8, "kv": 3001,
         "ragged": True, "q_heads": 16, "k_heads": 16, "dk": 64, "dv": 64, "page": 32,
         "window": 1024},
        # latent-attention heads expanded (192-wide keys, 128-wide values), two odd chunks
        {"name": "attn_mla777", "op": "attention", "new": 777, "seqs": 2, "kv": 2500,
         "ragged": False, "q_heads": 16, "k_heads": 16, "dk": 192, "dv": 128, "page": 64,
         "window": 0},
        # a small layer, two tokens, experts chosen within groups: latency
        {"name": "moe_small2", "op": "moe", "tokens": 2, "dim": 512, "inter": 256, "experts": 16,
         "top_k": 4, "groups": 4, "topk_groups": 2, "score": "sigmoid", "bias": True,
         "ue8m0": False},
        # one token through the 7168-wide layer with 2048-wide experts
        {"name": "moe_decode1", "op": "moe", "tokens": 1, "dim": 7168, "inter": 2048,
         "experts": 32, "top_k": 8, "groups": 8, "topk_groups": 4, "score": "sigmoid",
         "bias": True, "ue8m0": False},
        # a few sequences, power-of-two scales, plain softmax routing
        {"name": "moe_decode7_ue8m0", "op": "moe", "tokens": 7, "dim": 7168, "inter": 2048,
         "experts": 32, "top_k": 8, "groups": 1, "topk_groups": 1, "score": "softmax",
         "bias": False, "ue8m0": True},
        # a full decode batch: every expert is met
        {"name": "moe_decode64", "op": "moe", "tokens": 64, "dim": 7168, "inter": 2048,
         "experts": 32, "top_k": 8, "groups": 8, "topk_groups": 4, "score": "sigmoid",
         "bias": True, "ue8m0": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "attention", "attention", "moe"])
    if op == "norm_rope":
        dk, dv, rot, start = rng.choice([(64, 64, 64, 0), (64, 64, 32, 0), (128, 128, 128, 0),
                                         (128, 128, 64, 32), (192, 128, 64, 128)])
        k_heads = rng.choice([1, 2, 3, 4, 8, 16])
        return {"op": op, "tokens": _log_int(rng, 1, 4096), "q_heads": k_heads * rng.choice([1, 2, 3, 4]),
                "k_heads": k_heads, "dk": dk, "dv": dv, "rot": rot, "rot_start": start,
                "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.7,
                "page": rng.choice([1, 16, 48, 64])}
    if op == "attention":
        dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
        k_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 1, 3, 4, 7, 8]) if dk < 192 else 1
        new = 1 if rng.random() < 0.4 else _log_int(rng, 2, 1024)
        kv = _log_int(rng, max(64, new), 12000)
        seqs = max(1, min(_log_int(rng, 1, 48), int(1e9 / (new * kv * k_heads * group)),
                          int(1e9 / (kv * k_heads * 2 * (dk + dv)))))
        return {"op": op, "new": new, "seqs": seqs, "kv": kv, "ragged": rng.random() < 0.6,
                "q_heads": k_heads * group, "k_heads": k_heads, "dk": dk, "dv": dv,
                "page": rng.choice([16, 32, 48, 64, 128]),
                "window": rng.choice([0, 0, 0, 100, 2000])}
    experts = rng.choice([8, 16, 24, 32])
    groups = rng.choice([1, 1, 4, 8])
    topk_groups = 1 if groups == 1 else groups // 2
    softmax = rng.random() < 0.3
    return {"op": op, "tokens": _log_int(rng, 1, 64), "dim": BLOCK * _log_int(rng, 2, 56),
            "inter": BLOCK * _log_int(rng, 1, 16), "experts": experts,
            "top_k": rng.choice([1, 2, 4, min(8, experts // groups * topk_groups)]),
            "groups": groups, "topk_groups": topk_groups,
            "score": "softmax" if softmax else "sigmoid", "bias": not softmax,
            "ue8m0": rng.random() < 0.3}


# ------------------------------------------------------------------------------------ inputs

def _lengths(case):
    """New tokens and cached keys of every sequence (the same for every seed, so that `work` can
    count them): all alike, or spread over the whole range with the longest among them."""
    n, kv, seqs = case["new"], case["kv"], case["seqs"]
    if not case["ragged"]:
        return [n] * seqs, [kv] * seqs
    news, lens = [], []
    for b in range(seqs):
        f = ((b * 0.6180339887) % 1.0) if b else 1.0
        news.append(max(1, int(n * f * f)) if n > 1 else 1)
        lens.append(max(news[-1], int(kv * f)))
    return news, lens


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _cache(case, g, pages):
    """A paged cache with random contents."""
    k = _randn(g, pages, case["page"], case["k_heads"], case["dk"])
    v = _randn(g, pages, case["page"], case["k_heads"], case["dv"])
    return k, v


def _rope_tables(case, positions):
    half = case["rot"] // 2
    inv = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    ang = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "norm_rope":
        t, hq, hk, dk, dv = (case[n] for n in ("tokens", "q_heads", "k_heads", "dk", "dv"))
        pages = -(-t // case["page"]) + 3
        ck, cv = _cache(case, g, pages)
        cos, sin = _rope_tables(case, 2 * t + 100)
        # the projections' output in one row per token: q heads, then k heads, then v heads
        qkv = _randn(g, t, hq * dk + hk * dk + hk * dv, scale=1.5)
        q = qkv[:, :hq * dk].view(t, hq, dk)
        k = qkv[:, hq * dk:(hq + hk) * dk].view(t, hk, dk)
        v = qkv[:, (hq + hk) * dk:].view(t, hk, dv)
        slots = torch.randperm(pages * case["page"], generator=g, device="cuda")[:t].contiguous()
        positions = torch.randint(0, 2 * t + 100, (t,), generator=g, device="cuda",
                                  dtype=torch.int32)
        st = dict(q=q, k=k, v=v, ck=ck, cv=cv, cos=cos, sin=sin, slots=slots,
                  positions=positions, qw=None, kw=None)
        if case["norm"]:
            st["qw"] = (1.0 + 0.1 * torch.randn(dk, generator=g, device="cuda")).bfloat16()
            st["kw"] = (1.0 + 0.1 * torch.randn(dk, generator=g, device="cuda")).bfloat16()
    elif case["op"] == "attention":
        news, lens = _lengths(case)
        need = [-(-n // case["page"]) for n in lens]
        pages = sum(need) + 5
        ck, cv = _cache(case, g, pages)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu().numpy()
        table = np.zeros((len(lens), max(need)), dtype=np.int32)
        at = 0
        for b, c in enumerate(need):
            table[b, :c] = order[at:at + c]
            at += c
        # queries a little larger than unit: attention that is neither flat nor one key
        q = _randn(g, sum(news), case["q_heads"], case["dk"], scale=1.5)
        starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        st = dict(q=q, ck=ck, cv=cv, table=torch.from_numpy(table).cuda(),
                  q_start=torch.from_numpy(starts).cuda(),
                  kv_len=torch.tensor(lens, dtype=torch.int32).cuda(),
                  max_q=max(news), max_kv=max(lens))
    else:
        t, d, inter, e = (case[n] for n in ("tokens", "dim", "inter", "experts"))
        x = _randn(g, t, d)
        # one activation in a hundred stands far out
        far = torch.rand(t, d, generator=g, device="cuda") < 0.01
        x = torch.where(far, x * 20, x)
        router = _randn(g, e, d, scale=1.2 / math.sqrt(5 * d))
        bias = 0.05 * torch.randn(e, generator=g, device="cuda") if case["bias"] else None

        def weights(rows, cols):
            codes = torch.empty(e, rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
            for i in range(e):
                codes[i] = (torch.randn(rows, cols, generator=g, device="cuda") * 32).to(
                    torch.float8_e4m3fn)
            u = torch.rand(e, rows // BLOCK, cols // BLOCK, generator=g, device="cuda")
            s = torch.exp2(u * 2 - 1) / (32 * math.sqrt(cols))
            if case["ue8m0"]:
                s = torch.exp2(torch.round(torch.log2(s)))
            return codes, s

        w13, s13 = weights(2 * inter, d)
        w2, s2 = weights(d, inter)
        st = dict(x=x, router=router, bias=bias, w13=w13, s13=s13, w2=w2, s2=s2)
    st["case"] = case
    return st


# ------------------------------------------------------------------------------- plain forms

def _plain_norm_rope(st):
    c = st["case"]
    cos = st["cos"][st["positions"].long()][:, None]
    sin = st["sin"][st["positions"].long()][:, None]
    r0, r1 = c["rot_start"], c["rot_start"] + c["rot"]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        rot = x[..., r0:r1]
        if c["interleaved"]:
            a, b = rot[..., 0::2], rot[..., 1::2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = rot.chunk(2, -1)
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([x[..., :r0], turned, x[..., r1:]], -1).bfloat16()

    q = one(st["q"], st["qw"])
    st["ck"].flatten(0, 1)[st["slots"]] = one(st["k"], st["kw"])
    st["cv"].flatten(0, 1)[st["slots"]] = st["v"]
    return [q, st["ck"], st["cv"]]


def _plain_attention(st):
    c = st["case"]
    hk, dk, dv = c["k_heads"], c["dk"], c["dv"]
    grp = c["q_heads"] // hk
    seqs, mq, mk = c["seqs"], st["max_q"], st["max_kv"]
    q_start, kv_len = st["q_start"].long(), st["kv_len"].long()
    news = q_start[1:] - q_start[:-1]
    # keys, values and queries padded to the longest sequence
    k = st["ck"][st["table"].long()].flatten(1, 2)[:, :mk].float()
    v = st["cv"][st["table"].long()].flatten(1, 2)[:, :mk].float()
    i = torch.arange(mq, device="cuda")
    j = torch.arange(mk, device="cuda")
    rows = (q_start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][rows].float().view(seqs, mq, hk, grp, dk)
    s = q.permute(0, 2, 3, 1, 4).reshape(seqs, hk, grp * mq, dk) @ k.permute(0, 2, 3, 1)
    s = (s * dk ** -0.5).view(seqs, hk, grp, mq, mk)
    last = (kv_len - news)[:, None] + i
    open_ = j <= last[..., None]
    if c["window"]:
        open_ &= j > last[..., None] - c["window"]
    s = s.masked_fill_(~open_[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = (s - top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(seqs, hk, grp * mq, mk) @ v.permute(0, 2, 1, 3)).view(seqs, hk, grp, mq, dv)
    o = o / total
    lse = (top + total.log())[..., 0]
    real = i < news[:, None]
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, mq, c["q_heads"], dv)[real]
    lse = lse.permute(0, 3, 1, 2).reshape(seqs, mq, c["q_heads"])[real]
    return [o.bfloat16(), lse]


def _plain_quant(x, ue8m0):
    """e4m3 codes with one scale per 128 values, as the values that they stand for."""
    b = x.unflatten(-1, (-1, BLOCK))
    # a tensor as divisor: by a Python number torch multiplies with its reciprocal instead
    s = b.abs().amax(-1, keepdim=True).clamp(min=1e-4) / x.new_full((), 448.0)
    if ue8m0:
        # the next power of two: a carry out of the significand's bits
        s = ((s.view(torch.int32) + 0x7FFFFF) & 0x7F800000).view(torch.float32)
    return ((b / s).to(torch.float8_e4m3fn).float() * s).flatten(-2)


def _plain_route(st):
    c = st["case"]
    logits = st["x"].float() @ st["router"].float().T
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        ex = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = ex / ex.sum(-1, keepdim=True)
    choice = score if st["bias"] is None else score + st["bias"]
    if c["groups"] > 1:
        by = choice.unflatten(-1, (c["groups"], -1))
        if st["bias"] is None:
            best = by.amax(-1)
        else:
            best = by.sort(-1, descending=True)[0][..., :2].sum(-1)
        keep = torch.sort(best, dim=-1, descending=True, stable=True)[1][:, :c["topk_groups"]]
        mask = torch.zeros_like(best).scatter_(1, keep, 1.0)
        choice = by.masked_fill(mask[..., None] == 0, -math.inf).flatten(-2)
    ids = torch.sort(choice, dim=-1, descending=True, stable=True)[1][:, :c["top_k"]]
    w = score.gather(1, ids)
    if c["score"] == "sigmoid":
        w = w / w.sum(-1, keepdim=True)
    return w * 2.5, ids


def _plain_weight(codes, s):
    e, n, k = codes.shape
    w = codes.float().view(e, n // BLOCK, BLOCK, k // BLOCK, BLOCK)
    return (w * s[:, :, None, :, None]).view(e, n, k)


def _plain_moe(st):
    c = st["case"]
    inter = c["inter"]
    w, ids = _plain_route(st)
    x = _plain_quant(st["x"].float(), c["ue8m0"])
    if c["tokens"] * c["top_k"] <= c["experts"]:
        # few choices: the chosen experts' weights, one product for each token's choice
        chosen = ids.flatten()
        w13 = _plain_weight(st["w13"].view(torch.uint8)[chosen].view(torch.float8_e4m3fn),
                            st["s13"][chosen])
        gu = w13 @ x.repeat_interleave(c["top_k"], 0)[..., None]
        h = gu[:, :inter, 0]
        h = h / (1.0 + torch.exp(-h)) * gu[:, inter:, 0]
        w2 = _plain_weight(st["w2"].view(torch.uint8)[chosen].view(torch.float8_e4m3fn),
                           st["s2"][chosen])
        y = (w2 @ _plain_quant(h, c["ue8m0"])[..., None])[..., 0]
        y = (y.view(c["tokens"], c["top_k"], -1) * w[..., None]).sum(1)
    else:
        # every expert for every token, weighted by zero where it was not chosen
        dense = torch.zeros(c["tokens"], c["experts"], device="cuda").scatter_(1, ids, w)
        gu = x @ _plain_weight(st["w13"], st["s13"]).transpose(1, 2)
        h = gu[..., :inter]
        h = _plain_quant(h / (1.0 + torch.exp(-h)) * gu[..., inter:], c["ue8m0"])
        y = ((h * dense.T[..., None]) @ _plain_weight(st["w2"], st["s2"]).transpose(1, 2)).sum(0)
    return [y.bfloat16()]


def run(st):
    c = st["case"]
    if not own:
        return {"norm_rope": _plain_norm_rope, "attention": _plain_attention,
                "moe": _plain_moe}[c["op"]](st)
    import fp8_block_scaled_fp8bs_gb300 as f
    if c["op"] == "norm_rope":
        q = f.qk_norm_rope(st["q"], st["k"], st["cos"], st["sin"], st["positions"],
                           q_weight=st["qw"], k_weight=st["kw"], eps=1e-6,
                           rot_start=c["rot_start"], interleaved=c["interleaved"],
                           cache=f.PagedCache(st["ck"], st["cv"]), v=st["v"], slots=st["slots"])
        return [q, st["ck"], st["cv"]]
    if c["op"] == "attention":
        out, lse = f.paged_attention(st["q"], f.PagedCache(st["ck"], st["cv"]), st["table"],
                                     st["q_start"], st["kv_len"], causal=True, window=c["window"],
                                     max_q_len=st["max_q"], max_kv_len=st["max_kv"],
                                     return_lse=True)
        return [out, lse]
    return [f.moe_layer(st["x"], st["router"], st["w13"], st["s13"], st["w2"], st["s2"],
                        top_k=c["top_k"], bias=st["bias"], score=c["score"], groups=c["groups"],
                        topk_groups=c["topk_groups"], route_scale=2.5,
                        scale_fmt="ue8m0" if c["ue8m0"] else "fp32")]


# --------------------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "norm_rope":
        t, hq, hk, dk, dv = (case[n] for n in ("tokens", "q_heads", "k_heads", "dk", "dv"))
        elems = t * ((hq + hk) * dk + hk * dv)
        return {"bytes": 4 * elems + t * (4 * case["rot"] + 12),
                "flops": t * (hq + hk) * ((4 * dk if case["norm"] else 0) + 3 * case["rot"])}
    if case["op"] == "attention":
        news, lens = _lengths(case)
        pairs = 0
        for n, kv in zip(news, lens):
            open_ = np.arange(kv - n, kv, dtype=np.int64) + 1
            pairs += int((np.minimum(open_, case["window"]) if case["window"] else open_).sum())
        seen = sum(min(kv, n - 1 + case["window"]) if case["window"] else kv
                   for n, kv in zip(news, lens))
        hq, hk, dk, dv = (case[n] for n in ("q_heads", "k_heads", "dk", "dv"))
        return {"bytes": sum(news) * hq * (2 * (dk + dv) + 4) + seen * hk * 2 * (dk + dv),
                "flops": 2 * (dk + dv) * hq * pairs}
    t, d, inter, e, k = (case[n] for n in ("tokens", "dim", "inter", "experts", "top_k"))
    # experts that a random choice meets
    met = e * (1.0 - (1.0 - k / e) ** t)
    expert = 3 * d * inter * (1 + 4 / BLOCK ** 2)
    return {"bytes": int(met * expert) + 2 * e * d + 4 * t * d,
            "flops": 6 * t * k * d * inter + 2 * t * e * d}


# ------------------------------------------------------------------------------------- exact

def _exact_norm_rope(case, st):
    pos = st["positions"].long()
    turn = torch.complex(st["cos"].double()[pos], st["sin"].double()[pos])[:, None]
    outs = []
    for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        x = x.double()
        if w is not None:
            x = x / ((x ** 2).sum(-1, keepdim=True) / case["dk"] + 1e-6) ** 0.5 * w.double()
        else:
            x = x.clone()
        half = case["rot"] // 2
        idx = torch.arange(half, device="cuda") + 0
        lo = case["rot_start"] + (2 * idx if case["interleaved"] else idx)
        hi = lo + (1 if case["interleaved"] else half)
        z = torch.complex(x[..., lo], x[..., hi]) * turn
        x[..., lo], x[..., hi] = z.real, z.imag
        outs.append(x)
    ck, cv = st["ck"].double(), st["cv"].double()
    page = case["page"]
    ck[st["slots"] // page, st["slots"] % page] = outs[1]
    cv[st["slots"] // page, st["slots"] % page] = st["v"].double()
    return [outs[0], ck, cv]


def _exact_attention(case, st):
    news, lens = _lengths(case)
    hq, hk, dk, dv = (case[n] for n in ("q_heads", "k_heads", "dk", "dv"))
    out = torch.zeros(sum(news), hq, dv, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(news), hq, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, kv) in enumerate(zip(news, lens)):
        at = torch.arange(kv, device="cuda")
        page = st["table"][b].long()[at // case["page"]]
        k, v = st["ck"][page, at % case["page"]], st["cv"][page, at % case["page"]]
        for r0 in range(0, n, 1024):
            r1 = min(n, r0 + 1024)
            here = torch.arange(kv - n + r0, kv - n + r1, device="cuda")[:, None]
            shut = at > here
            if case["window"]:
                shut |= at <= here - case["window"]
            for h in range(hk):
                heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
                q = st["q"][t0 + r0:t0 + r1, heads].double()
                s = torch.einsum("nhd,kd->hnk", q, k[:, h].double()) / math.sqrt(dk)
                s[:, shut] = -math.inf
                total = torch.logsumexp(s, -1)
                o = torch.einsum("hnk,kd->nhd", torch.exp(s - total[..., None]), v[:, h].double())
                out[t0 + r0:t0 + r1, heads] = o
                lse[t0 + r0:t0 + r1, heads] = total.T
        t0 += n
    return [out, lse]


def _power_of_two(e):
    """2^e in binary64 from its bits (torch's pow and ldexp are not exact on every device)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_quant(x, ue8m0):
    """Block quantisation by its definition: the scale and the quotient are binary32 numbers, the
    code is the nearest e4m3 number (ties to even), found here by rounding the significand."""
    x = x.float().double().unflatten(-1, (-1, BLOCK))
    s = (x.abs().amax(-1, keepdim=True).clamp(min=float(np.float32(1e-4))) / 448.0).float().double()
    if ue8m0:
        m, e = torch.frexp(s)
        s = _power_of_two(torch.where(m > 0.5, e, e - 1))
    v = (x / s).float().double()
    _, e = torch.frexp(v)
    ulp = _power_of_two((e - 4).clamp(min=-9))
    return ((torch.round(v / ulp) * ulp).clamp(-448, 448) * s).flatten(-2)


def _exact_moe(case, st):
    x = st["x"].double()
    t, inter = case["tokens"], case["inter"]
    logits = x @ st["router"].double().T
    score = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits, -1)
    choice = score + (0 if st["bias"] is None else st["bias"].double())
    xq = _exact_quant(x, case["ue8m0"])
    picked = []
    for i, row in enumerate(choice.cpu().numpy()):
        by = row.reshape(case["groups"], -1)
        top = np.sort(by, 1)[:, ::-1]
        rank = top[:, 0] if st["bias"] is None else top[:, :2].sum(1)
        keep = np.argsort(-rank, kind="stable")[:case["topk_groups"]]
        shut = np.full_like(by, -np.inf)
        shut[keep] = by[keep]
        picked.append(np.argsort(-shut.ravel(), kind="stable")[:case["top_k"]])
    picked = torch.from_numpy(np.stack(picked)).cuda()
    w = torch.take_along_dim(score, picked, 1)
    if case["score"] == "sigmoid":
        w = w / w.sum(1, keepdim=True)
    w = w * 2.5
    y = torch.zeros_like(x)

    def product(a, codes, s):
        full = s.double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
        return a @ (codes.double() * full).T

    for e in range(case["experts"]):
        rows, slot = torch.where(picked == e)
        if len(rows):
            gu = product(xq[rows], st["w13"][e], st["s13"][e])
            h = gu[:, :inter] * torch.sigmoid(gu[:, :inter]) * gu[:, inter:]
            y[rows] += w[rows, slot][:, None] * product(_exact_quant(h, case["ue8m0"]),
                                                        st["w2"][e], st["s2"][e])
    return [y]


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "attention": _exact_attention,
            "moe": _exact_moe}[case["op"]](case, st)
