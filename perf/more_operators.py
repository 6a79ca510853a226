"""Cases of the operators that keep a decoder layer's activations and cache in 8 bits, for measurement:

  rms_norm          the residual's addition, RMS norm and the e4m3 codes of the next product
  qk_norm_rope      norms of queries and keys per head, position rotation, write into a cache of e4m3 codes
  paged_attention   attention of new tokens over such a cache: one scale per page and head

`run` computes each in its plain form (elementary torch operations in 32 bits) or, with `own`,
through the package's entry points; `exact` computes it from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # a decode step of five sequences through the 7168-wide layer: codes for the product and, for a
        # router, bf16
        {"name": "norm_decode5", "op": "norm", "tokens": 5, "dim": 7168, "residual": True,
         "quant": "fp32", "norm": True},
        # a long prefill chunk of the same layer
        {"name": "norm_chunk8192", "op": "norm", "tokens": 8192, "dim": 7168, "residual": True,
         "quant": "fp32", "norm": False},
        # the norm of latent queries (1536 channels), power-of-two scales, no residual
        {"name": "norm_latent333", "op": "norm", "tokens": 333, "dim": 1536, "residual": False,
         "quant": "ue8m0", "norm": False},
        # a decode step of 61 sequences: every token goes into the middle of a page
        {"name": "write_decode61", "op": "write", "new": 1, "seqs": 61, "ragged": False, "q_heads": 32,
         "k_heads": 8, "dk": 128, "dv": 128, "rot": 128, "rot_start": 0, "interleaved": False,
         "norm": True, "page": 64},
        # a long prefill chunk, begun in the middle of a page
        {"name": "write_chunk8192", "op": "write", "new": 8192, "seqs": 1, "ragged": False, "q_heads": 32,
         "k_heads": 8, "dk": 128, "dv": 128, "rot": 128, "rot_start": 0, "interleaved": False,
         "norm": True, "page": 64},
        # expanded latent-attention heads, chunks of several sequences: the last 64 channels rotate, no norm
        {"name": "write_mla4x300", "op": "write", "new": 300, "seqs": 4, "ragged": True, "q_heads": 16,
         "k_heads": 16, "dk": 192, "dv": 128, "rot": 64, "rot_start": 128, "interleaved": True,
         "norm": False, "page": 16},
        # a few short conversations: latency
        {"name": "attn_decode3_short", "op": "attention", "new": 1, "seqs": 3, "kv": 301,
         "ragged": True, "q_heads": 32, "k_heads": 8, "dk": 128, "dv": 128, "page": 16, "window": 0},
        # one token of one long conversation: the split over the key axis
        {"name": "attn_decode1_32k", "op": "attention", "new": 1, "seqs": 1, "kv": 32785,
         "ragged": False, "q_heads": 32, "k_heads": 8, "dk": 128, "dv": 128, "page": 64, "window": 0},
        # a decode batch of conversations of all lengths
        {"name": "attn_decode64_ragged", "op": "attention", "new": 1, "seqs": 64, "kv": 8192,
         "ragged": True, "q_heads": 64, "k_heads": 8, "dk": 128, "dv": 128, "page": 16, "window": 0},
        # the second half of a long prompt, prefilled as one chunk over the cached first half
        {"name": "attn_chunk4096", "op": "attention", "new": 4096, "seqs": 1, "kv": 8192,
         "ragged": False, "q_heads": 32, "k_heads": 8, "dk": 128, "dv": 128, "page": 64, "window": 0},
        # chunks and decodes mixed in one batch, sliding window, as many key heads as query heads
        {"name": "attn_mixed8_window", "op": "attention", "new": 300, "seqs": 8, "kv": 3001,
         "ragged": True, "q_heads": 16, "k_heads": 16, "dk": 64, "dv": 64, "page": 32, "window": 1024},
        # expanded latent-attention heads, three drafted tokens a sequence
        {"name": "attn_mla24x3", "op": "attention", "new": 3, "seqs": 24, "kv": 5000,
         "ragged": True, "q_heads": 16, "k_heads": 16, "dk": 192, "dv": 128, "page": 64, "window": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "write", "attention", "attention"])
    if op == "norm":
        dim = BLOCK * _log_int(rng, 2, 64)
        # (power-of-two scales: a decode batch's worth of tokens)
        quant = rng.choice(["fp32", "fp32", "none", "ue8m0"])
        most = 4096 if quant != "ue8m0" else max(2, (1 << 20) // dim)
        return {"op": op, "tokens": _log_int(rng, 1, most), "dim": dim, "residual": rng.random() < 0.6,
                "quant": quant, "norm": quant == "none" or rng.random() < 0.4}
    if op == "write":
        dk, dv, rot, start = rng.choice([(64, 64, 64, 0), (64, 64, 32, 0), (128, 128, 128, 0),
                                         (128, 128, 64, 32), (192, 128, 64, 128)])
        k_heads = rng.choice([1, 2, 3, 4, 8, 16])
        new = 1 if rng.random() < 0.4 else _log_int(rng, 2, 2048)
        return {"op": op, "new": new, "seqs": _log_int(rng, 1, max(1, min(200, 4096 // new))),
                "ragged": rng.random() < 0.5, "q_heads": k_heads * rng.choice([1, 2, 3, 4]),
                "k_heads": k_heads, "dk": dk, "dv": dv, "rot": rot, "rot_start": start,
                "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.7,
                "page": rng.choice([16, 32, 48, 64, 128])}
    dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
    k_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 1, 3, 4, 7, 8, 16])
    new = 1 if rng.random() < 0.5 else _log_int(rng, 2, 1024)
    kv = _log_int(rng, max(64, new), 12000)
    seqs = max(1, min(_log_int(rng, 1, 48), int(8e8 / (new * kv * k_heads * group)),
                      int(1e9 / (kv * k_heads * 2 * (dk + dv)))))
    return {"op": op, "new": new, "seqs": seqs, "kv": kv, "ragged": rng.random() < 0.6,
            "q_heads": k_heads * group, "k_heads": k_heads, "dk": dk, "dv": dv,
            "page": rng.choice([16, 32, 48, 64, 128]), "window": rng.choice([0, 0, 0, 100, 2000])}


# ------------------------------------------------------------------------------------ inputs

def _lengths(case):
    """New tokens and cached keys of every sequence (the same for every seed, so that `work` can
    count them): all alike, or spread over the whole range with the longest among them. What is
    written begins anywhere in a page."""
    n, seqs = case["new"], case["seqs"]
    kv = case.get("kv")
    news, lens = [], []
    for b in range(seqs):
        f = ((b * 0.6180339887) % 1.0) if b and case["ragged"] else 1.0
        news.append(max(1, int(n * f * f)) if n > 1 else 1)
        if kv is None:
            lens.append(news[-1] + (37 + 29 * b) % (2 * case["page"]))
        else:
            lens.append(max(news[-1], int(kv * f)))
    return news, lens


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _power_above(x):
    """The smallest power of two that is at least x: a carry out of the significand's bits."""
    return ((x.view(torch.int32) + 0x7FFFFF) & 0x7F800000).view(torch.float32)


def _scale_of(amax):
    # (a tensor as divisor: by a Python number torch multiplies with its reciprocal instead)
    return _power_above(amax.clamp(min=1e-4) / amax.new_full((), 448.0))


def _codes(case, g, pages, d, spread):
    """Codes [pages, page, heads, d] and scales [pages, heads] of normal values whose size differs
    from page to page and head to head by 2^+-spread."""
    codes = torch.empty(pages, case["page"], case["k_heads"], d, dtype=E4M3, device="cuda")
    scales = torch.empty(pages, case["k_heads"], device="cuda")
    for p in range(0, pages, 4096):
        q = min(pages, p + 4096)
        x = torch.randn(q - p, case["page"], case["k_heads"], d, generator=g, device="cuda")
        size = torch.rand(q - p, 1, case["k_heads"], 1, generator=g, device="cuda") * 2 - 1
        x *= torch.exp2(spread * size)
        s = _scale_of(x.abs().amax((1, 3)))
        codes[p:q] = (x / s[:, None, :, None]).to(E4M3)
        scales[p:q] = s
    return codes, scales


def _tables(case, g, lens):
    """Pages of every sequence, in random order, in one pool with a few spare ones."""
    need = [-(-n // case["page"]) for n in lens]
    pages = sum(need) + 5
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu().numpy()
    table = np.zeros((len(lens), max(need)), dtype=np.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    return pages, table


def _rope_tables(case, positions):
    half = case["rot"] // 2
    inv = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    ang = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "norm":
        t, d = case["tokens"], case["dim"]
        x = _randn(g, t, d)
        st = dict(x=x, r=None, w=(1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).bfloat16())
        if case["residual"]:
            # a residual stream: larger than what a layer adds, a few channels far out
            far = torch.rand(d, generator=g, device="cuda") < 0.01
            st["r"] = torch.where(far, _randn(g, t, d, scale=40.0), _randn(g, t, d, scale=4.0))
    elif case["op"] == "write":
        news, lens = _lengths(case)
        t = sum(news)
        hq, hk, dk, dv = (case[n] for n in ("q_heads", "k_heads", "dk", "dv"))
        pages, table = _tables(case, g, lens)
        ck, sk = _codes(case, g, pages, dk, 1.0)
        cv, sv = _codes(case, g, pages, dv, 1.0)
        # the projections' output in one row per token: q heads, then k heads, then v heads
        qkv = _randn(g, t, hq * dk + hk * dk + hk * dv, scale=1.5)
        at = np.concatenate([np.arange(n - m, n) for m, n in zip(news, lens)])
        seq = np.repeat(np.arange(len(news)), news)
        slots = table[seq, at // case["page"]].astype(np.int64) * case["page"] + at % case["page"]
        cos, sin = _rope_tables(case, max(lens) + 100)
        st = dict(q=qkv[:, :hq * dk].view(t, hq, dk),
                  k=qkv[:, hq * dk:(hq + hk) * dk].view(t, hk, dk),
                  v=qkv[:, (hq + hk) * dk:].view(t, hk, dv),
                  ck=ck, cv=cv, sk=sk, sv=sv, cos=cos, sin=sin, slots=torch.from_numpy(slots).cuda(),
                  positions=torch.from_numpy(at.astype(np.int32)).cuda(), qw=None, kw=None)
        if case["norm"]:
            st["qw"] = (1.0 + 0.1 * torch.randn(dk, generator=g, device="cuda")).bfloat16()
            st["kw"] = (1.0 + 0.1 * torch.randn(dk, generator=g, device="cuda")).bfloat16()
    else:
        news, lens = _lengths(case)
        pages, table = _tables(case, g, lens)
        ck, sk = _codes(case, g, pages, case["dk"], 0.5)
        cv, sv = _codes(case, g, pages, case["dv"], 2.0)
        # queries a little larger than unit: attention that is neither flat nor one key
        q = _randn(g, sum(news), case["q_heads"], case["dk"], scale=1.5)
        starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        st = dict(q=q, ck=ck, cv=cv, sk=sk, sv=sv, table=torch.from_numpy(table).cuda(),
                  q_start=torch.from_numpy(starts).cuda(),
                  kv_len=torch.tensor(lens, dtype=torch.int32).cuda(),
                  max_q=max(news), max_kv=max(lens))
    st["case"] = case
    return st


# ------------------------------------------------------------------------------- plain forms

def _plain_norm(st):
    c = st["case"]
    h = st["x"]
    outs = []
    if c["residual"]:
        h = (h.float() + st["r"].float()).bfloat16()
        outs.append(h)
    x = h.float()
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * st["w"].float()
    if c["norm"]:
        outs.append(n.bfloat16())
    if c["quant"] != "none":
        b = n.unflatten(-1, (-1, BLOCK))
        s = b.abs().amax(-1, keepdim=True).clamp(min=1e-4) / n.new_full((), 448.0)
        if c["quant"] == "ue8m0":
            s = _power_above(s)
        outs += [(b / s).to(E4M3).flatten(-2), s[..., 0]]
    return outs


def _plain_rows(c, x, w, cos, sin):
    """Norm and rotation of rows [T, heads, d], in 32 bits."""
    r0, r1 = c["rot_start"], c["rot_start"] + c["rot"]
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
    return torch.cat([x[..., :r0], turned, x[..., r1:]], -1)


def _plain_write(st):
    c = st["case"]
    cos = st["cos"][st["positions"].long()][:, None]
    sin = st["sin"][st["positions"].long()][:, None]
    q = _plain_rows(c, st["q"], st["qw"], cos, sin).bfloat16()
    page, off = st["slots"] // c["page"], st["slots"] % c["page"]
    first = torch.zeros(st["sk"].shape[0], dtype=torch.bool, device="cuda")
    first[page[off == 0]] = True
    for x, codes, scale in ((_plain_rows(c, st["k"], st["kw"], cos, sin), st["ck"], st["sk"]),
                            (st["v"].float(), st["cv"], st["sv"])):
        need = torch.zeros_like(scale).index_reduce_(0, page, _scale_of(x.abs().amax(-1)), "amax")
        old = scale.masked_fill(first[:, None], 0.0)
        new = torch.where(need > 0, torch.maximum(old, need), scale)
        keep = torch.where((need > 0) & (old > 0), old / new, torch.ones_like(old))
        codes.copy_((codes.float() * keep[:, None, :, None]).to(E4M3))
        codes.view(torch.uint8).flatten(0, 1)[st["slots"]] = (x / new[page][..., None]).to(
            E4M3).view(torch.uint8)
        scale.copy_(new)
    return [q, st["ck"], st["sk"], st["cv"], st["sv"]]


def _plain_attention(st):
    c = st["case"]
    hk, dk, dv = c["k_heads"], c["dk"], c["dv"]
    grp = c["q_heads"] // hk
    seqs, mq, mk = c["seqs"], st["max_q"], st["max_kv"]
    q_start, kv_len = st["q_start"].long(), st["kv_len"].long()
    news = q_start[1:] - q_start[:-1]

    def gathered(codes, scale):
        # keys or values padded to the longest sequence
        t = st["table"].long()
        x = codes.view(torch.uint8)[t].view(E4M3).float() * scale[t][:, :, None, :, None]
        return x.flatten(1, 2)[:, :mk]

    k, v = gathered(st["ck"], st["sk"]), gathered(st["cv"], st["sv"])
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


def run(st):
    c = st["case"]
    if not own:
        return {"norm": _plain_norm, "write": _plain_write, "attention": _plain_attention}[c["op"]](st)
    import fp8_block_scaled_fp8bs_gb300 as f
    if c["op"] == "norm":
        quant = None if c["quant"] == "none" else c["quant"]
        got = f.rms_norm(st["x"], st["w"], eps=1e-6, residual=st["r"], quant=quant, norm=c["norm"])
        return [x for x in (got.h if c["residual"] else None, got.n, got.y, got.s) if x is not None]
    cache = f.PagedCacheFp8(st["ck"], st["cv"], st["sk"], st["sv"])
    if c["op"] == "write":
        q = f.qk_norm_rope(st["q"], st["k"], st["cos"], st["sin"], st["positions"],
                           q_weight=st["qw"], k_weight=st["kw"], eps=1e-6,
                           rot_start=c["rot_start"], interleaved=c["interleaved"], cache=cache,
                           v=st["v"], slots=st["slots"])
        return [q, st["ck"], st["sk"], st["cv"], st["sv"]]
    out, lse = f.paged_attention(st["q"], cache, st["table"], st["q_start"], st["kv_len"],
                                 causal=True, window=c["window"], max_q_len=st["max_q"],
                                 max_kv_len=st["max_kv"], return_lse=True)
    return [out, lse]


# --------------------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "norm":
        elems = case["tokens"] * case["dim"]
        each = 2 + 4 * case["residual"] + 2 * case["norm"]
        each += 0 if case["quant"] == "none" else 1 + 4 / BLOCK
        return {"bytes": int(elems * each) + 2 * case["dim"],
                "flops": elems * (4 + case["residual"] + (0 if case["quant"] == "none" else 2))}
    news, lens = _lengths(case)
    hq, hk, dk, dv = (case[n] for n in ("q_heads", "k_heads", "dk", "dv"))
    if case["op"] == "write":
        t = sum(news)
        pages = sum((n - 1) // case["page"] - (n - m) // case["page"] + 1 for m, n in zip(news, lens))
        return {"bytes": t * (4 * hq * dk + 3 * hk * (dk + dv) + 4 * case["rot"] + 12) + 8 * pages * hk,
                "flops": t * ((hq + hk) * ((4 * dk if case["norm"] else 0) + 3 * case["rot"]) +
                              2 * hk * (dk + dv))}
    pairs = 0
    for n, kv in zip(news, lens):
        open_ = np.arange(kv - n, kv, dtype=np.int64) + 1
        pairs += int((np.minimum(open_, case["window"]) if case["window"] else open_).sum())
    seen = sum(min(kv, n - 1 + case["window"]) if case["window"] else kv for n, kv in zip(news, lens))
    return {"bytes": sum(news) * hq * (2 * (dk + dv) + 4) +
            seen * hk * (dk + dv) + 8 * (seen // case["page"]) * hk,
            "flops": 2 * (dk + dv) * hq * pairs}


# ------------------------------------------------------------------------------------- exact

def _power_of_two(e):
    """2^e in binary64 from its bits (torch's pow and ldexp are not exact on every device)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_power_above(s):
    m, e = torch.frexp(s)
    return _power_of_two(torch.where(m > 0.5, e, e - 1))


def _exact_e4m3(v):
    """The nearest e4m3 number (ties to even), by rounding the significand."""
    _, e = torch.frexp(v)
    ulp = _power_of_two((e - 4).clamp(min=-9))
    return (torch.round(v / ulp) * ulp).clamp(-448, 448)


def _exact_norm(case, st):
    h, outs = st["x"].double(), []
    if case["residual"]:
        # the stored stream: the sum of two bf16 numbers, rounded once
        h = (h + st["r"].double()).bfloat16().double()
        outs.append(h)
    n = h / (h.pow(2).sum(-1, keepdim=True) / case["dim"] + 1e-6).sqrt() * st["w"].double()
    if case["norm"]:
        outs.append(n)
    if case["quant"] != "none":
        b = n.reshape(case["tokens"], -1, BLOCK)
        s = b.abs().max(-1)[0].clamp(min=float(np.float32(1e-4))) / 448
        if case["quant"] == "ue8m0":
            s = _exact_power_above(s)
        outs += [_exact_e4m3(b / s[..., None]).reshape(n.shape), s]
    return outs


def _exact_write(case, st):
    pos = st["positions"].long()
    turn = torch.complex(st["cos"].double()[pos], st["sin"].double()[pos])[:, None]
    rows = []
    for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        x = x.double()
        if w is not None:
            x = x / ((x ** 2).sum(-1, keepdim=True) / case["dk"] + 1e-6) ** 0.5 * w.double()
        else:
            x = x.clone()
        half = case["rot"] // 2
        idx = torch.arange(half, device="cuda")
        lo = case["rot_start"] + (2 * idx if case["interleaved"] else idx)
        hi = lo + (1 if case["interleaved"] else half)
        z = torch.complex(x[..., lo], x[..., hi]) * turn
        x[..., lo], x[..., hi] = z.real, z.imag
        rows.append(x)
    outs = [rows[0]]
    news, lens = _lengths(case)
    slots = st["slots"].cpu().numpy()
    for x, codes, scale in ((rows[1], st["ck"], st["sk"]), (st["v"].double(), st["cv"], st["sv"])):
        codes, scale = codes.double(), scale.double()
        t = 0
        while t < len(slots):
            # the run of tokens that go to one page
            page, off = divmod(int(slots[t]), case["page"])
            end = t + 1
            while end < len(slots) and slots[end] == slots[end - 1] + 1 and slots[end] // case["page"] == page:
                end += 1
            run_ = x[t:end]
            s = _exact_power_above(run_.abs().amax((0, 2)).clamp(min=1e-4) / 448)
            if off:
                s = torch.maximum(s, scale[page])
                codes[page] = _exact_e4m3(codes[page] * (scale[page] / s)[:, None])
            codes[page, off:off + end - t] = _exact_e4m3(run_ / s[:, None])
            scale[page] = s
            t = end
        outs += [codes, scale]
    return outs


def _exact_attention(case, st):
    news, lens = _lengths(case)
    hq, hk, dk, dv = (case[n] for n in ("q_heads", "k_heads", "dk", "dv"))
    out = torch.zeros(sum(news), hq, dv, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(news), hq, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, kv) in enumerate(zip(news, lens)):
        at = torch.arange(kv, device="cuda")
        page = st["table"][b].long()[at // case["page"]]
        for r0 in range(0, n, 1024):
            r1 = min(n, r0 + 1024)
            here = torch.arange(kv - n + r0, kv - n + r1, device="cuda")[:, None]
            shut = at > here
            if case["window"]:
                shut |= at <= here - case["window"]
            for h in range(hk):
                heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
                k = st["ck"].view(torch.uint8)[page, at % case["page"], h].view(E4M3).double()
                v = st["cv"].view(torch.uint8)[page, at % case["page"], h].view(E4M3).double()
                k = k * st["sk"].double()[page, h][:, None]
                v = v * st["sv"].double()[page, h][:, None]
                q = st["q"][t0 + r0:t0 + r1, heads].double()
                s = torch.einsum("nhd,kd->hnk", q, k) / math.sqrt(dk)
                s[:, shut] = -math.inf
                total = torch.logsumexp(s, -1)
                o = torch.einsum("hnk,kd->nhd", torch.exp(s - total[..., None]), v)
                out[t0 + r0:t0 + r1, heads] = o
                lse[t0 + r0:t0 + r1, heads] = total.T
        t0 += n
    return [out, lse]


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "write": _exact_write, "attention": _exact_attention}[case["op"]](case, st)
