"""Measured cases of the operators around the attention kernels: the paged cache's plan, the
queries' and keys' norm with the position rotation, and the cache held in 4 bits.

Four operators, two cases at least for each:

  plan      block tables and slot maps built on the device from request lengths (paged_plan)
  rope      RMS norm of each query and key head with the position rotation in the same pass:
            forward, backward, and the serving form that also writes the rows of k and v into
            their pages (qk_norm_rope, qk_norm_rope_bwd, qk_norm_rope_append)
  kv4       rows of k and v written into a 4-bit paged cache and read back from it
            (kv4_append, kv4_gather)
  decode4   attention of one to sixteen new queries over that cache (attn_decode_kv4)

``own`` False computes them in elementary torch operations, in 32 bits (64 where a value lies
next to a border); True calls the library.

A row of the 4-bit cache is D/2 + 4 bytes: element 2i of the row is the low nibble of byte i and
element 2i + 1 its high one; then two bf16 values, the step s and the minimum m of the row. The
row stands for s * code + m, with m the row's smallest value, s = bf16((max - min) / 15) and
code = round_half_even((x - m) * r) for r = 1 / s rounded to 32 bits.
"""
import random

import torch

own = False

_DEV = "cuda"


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 64 requests whose caches hold 4096 to 32768 tokens: one new token each
        {"name": "plan step 64", "op": "plan", "S": 64, "lo": 4096, "hi": 32768, "new_lo": 1, "new_hi": 1,
         "drop": 0, "page": 64},
        # a large mixed step: chunks of 0 to 255 tokens for 1024 requests, some of them finished
        # or rolled back behind a rejected draft
        {"name": "plan mixed 1024", "op": "plan", "S": 1024, "lo": 1, "hi": 2048, "new_lo": 0, "new_hi": 255,
         "drop": 5, "page": 16},
        # training at the shape of the grouped-query prefill workload, from the fused projection
        {"name": "rope forward 4x4096", "op": "rope", "way": "forward", "B": 4, "T": 4096, "Hq": 32, "Hkv": 8,
         "D": 128, "rot": 128, "pairs": "halves", "norm": True},
        {"name": "rope backward 4x4096", "op": "rope", "way": "backward", "B": 4, "T": 4096, "Hq": 32, "Hkv": 8,
         "D": 128, "rot": 128, "pairs": "halves", "norm": True},
        # odd length, six heads over two, half of each head rotated, neighbours paired
        {"name": "rope backward 3x577", "op": "rope", "way": "backward", "B": 3, "T": 577, "Hq": 6, "Hkv": 2,
         "D": 64, "rot": 32, "pairs": "neighbours", "norm": True},
        # one decode step of 64 requests: rotate, and write k and v into their pages
        {"name": "rope append 64", "op": "rope", "way": "append", "N": 64, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "pairs": "halves", "norm": True, "page": 64},
        # the chunked prefill workload's query tokens
        {"name": "rope append 35197", "op": "rope", "way": "append", "N": 35197, "Hq": 32, "Hkv": 8, "D": 128,
         "rot": 128, "pairs": "halves", "norm": True, "page": 64},
        # cache writes in 4 bits and their reading back: a decode step, and a prefill's tokens
        {"name": "kv4 rows 64", "op": "kv4", "N": 64, "Hkv": 8, "D": 128, "page": 64},
        {"name": "kv4 rows 35197", "op": "kv4", "N": 35197, "Hkv": 8, "D": 128, "page": 64},
        # a single request: few rows, latency counts
        {"name": "decode4 1x4099", "op": "decode4", "B": 1, "lo": 4099, "hi": 4099, "Hq": 32, "Hkv": 8, "D": 128,
         "Tq": 1, "page": 64, "window": 0},
        # the paged decode workload: 64 requests of 4096 to 32768 keys
        {"name": "decode4 64 ragged", "op": "decode4", "B": 64, "lo": 4096, "hi": 32768, "Hq": 32, "Hkv": 8, "D": 128,
         "Tq": 1, "page": 64, "window": 0},
        # verification chunks of four tokens in a sliding window, small pages, short heads
        {"name": "decode4 chunk window", "op": "decode4", "B": 37, "lo": 1, "hi": 8191, "Hq": 16, "Hkv": 4, "D": 64,
         "Tq": 4, "page": 16, "window": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


_HEADS = [(32, 8), (16, 16), (32, 1), (8, 2), (6, 2), (16, 4)]


def draw(rng):
    op = rng.choice(["plan", "forward", "backward", "append", "kv4", "decode4", "decode4"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        hi = _log(rng, 1, 16384)
        S = _log(rng, 1, 1024)
        return {"op": "plan", "S": S, "lo": rng.randint(0, hi), "hi": hi, "new_lo": rng.randint(0, 1),
                "new_hi": _log(rng, 1, max(1, 131072 // S)), "drop": rng.choice([0, 0, 4, 9]), "page": page}
    Hq, Hkv = rng.choice(_HEADS)
    D = rng.choice([64, 128])
    if op in ("forward", "backward", "append"):
        c = {"op": "rope", "way": op, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rng.choice([D, D, D // 2, D // 4]),
             "pairs": rng.choice(["halves", "neighbours"]), "norm": rng.random() < 0.8}
        if op == "append":
            return dict(c, N=_log(rng, 1, 32768), page=page)
        return dict(c, B=rng.randint(1, 4), T=_log(rng, 1, 4096))
    if op == "kv4":
        return {"op": "kv4", "N": _log(rng, 1, 32768), "Hkv": Hkv, "D": D, "page": page}
    hi = _log(rng, 1, 32768)
    B = min(_log(rng, 1, 64), max(1, (64 * 32768 * 1024) // (hi * Hkv * D)))
    return {"op": "decode4", "B": B, "lo": rng.randint(max(1, hi // 8), hi), "hi": hi, "Hq": Hq, "Hkv": Hkv, "D": D,
            "Tq": rng.choice([1, 1, 1, 2, 4]), "page": page,
            "window": rng.choice([0, 0, 0, _log(rng, 16, 4096)])}


def _ints(case, word, n, lo, hi):
    """n whole numbers in [lo, hi], of the case alone: its lengths are the same for every seed."""
    r = random.Random("%s %s %d" % (sorted((k, v) for k, v in case.items() if k != "name"), word, n))
    return [r.randint(lo, hi) for _ in range(n)]


def _plan_lengths(case):
    """(held, keep, new) of each request. One in `drop` rolls back or ends."""
    S = case["S"]
    held = _ints(case, "held", S, case["lo"], case["hi"])
    new = _ints(case, "new", S, case["new_lo"], case["new_hi"])
    keep = list(held)
    if case["drop"]:
        for s, (what, part) in enumerate(zip(_ints(case, "what", S, 0, 2 * case["drop"] - 1),
                                             _ints(case, "part", S, 0, 1 << 20))):
            if what == 0:  # finished: every page goes back
                keep[s], new[s] = 0, 0
            elif what == 1:  # rolled back behind a rejected draft
                keep[s] = max(0, held[s] - part % 17)
    return held, keep, new


def _decode_lengths(case):
    return _ints(case, "keys", case["B"], case["lo"], case["hi"])


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=_DEV)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=_DEV).to(torch.bfloat16)


def _perm(g, n):
    return torch.randperm(n, generator=g, device=_DEV).to(torch.int32)


def _table(positions, rot):
    """cos and sin of every position's angles, from 64 bits."""
    f = torch.arange(rot // 2, dtype=torch.float64, device=_DEV) * (2.0 / rot)
    a = torch.arange(positions, dtype=torch.float64, device=_DEV)[:, None] * (10000.0 ** -f)
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "plan":
        return _prepare_plan(case, g)
    if case["op"] == "rope":
        return _prepare_rope(case, g)
    if case["op"] == "kv4":
        N, Hkv, D, page = case["N"], case["Hkv"], case["D"], case["page"]
        pages = (N + page - 1) // page + 3
        s = dict(case, k=_normal(g, N, Hkv, D), v=_normal(g, N, Hkv, D), slots=_slots(g, N, page, pages))
        for p in ("k_pool", "v_pool"):
            s[p] = _quantise(_normal(g, pages, Hkv, page, D))
        return s
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    lens = _decode_lengths(case)
    max_pages = (max(lens) + page - 1) // page
    held = [(n + page - 1) // page for n in lens]
    pages = sum(held) + 2
    order = _perm(g, pages)
    table = torch.zeros(B, max_pages, dtype=torch.int32, device=_DEV)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    s = dict(case, q=_normal(g, B, case["Hq"], case["Tq"], D), table=table, lens=_i32(lens), longest=max(lens))
    channel = 1.0 + 0.2 * torch.randn(Hkv, 1, D, generator=g, device=_DEV)
    for p in ("k_pool", "v_pool"):
        pool = torch.empty(pages, Hkv, page, D // 2 + 4, dtype=torch.uint8, device=_DEV)
        step = max(1, (1 << 26) // (Hkv * page * D))
        for i in range(0, pages, step):
            n = min(step, pages - i)
            pool[i:i + n] = _quantise((torch.randn(n, Hkv, page, D, generator=g, device=_DEV) * channel).bfloat16())
        s[p] = pool
    return s


def _slots(g, N, page, pages):
    """N rows of a pool: tokens in order, in pages of any order."""
    t = torch.arange(N, device=_DEV)
    return (_perm(g, pages)[t // page].long() * page + t % page).to(torch.int32)


def _prepare_plan(case, g):
    held, keep, new = _plan_lengths(case)
    page = case["page"]
    pages_of = lambda n: (n + page - 1) // page  # noqa: E731
    most = max(max(k + n for k, n in zip(keep, new)), max(held), 1)
    max_pages = pages_of(most)
    used = sum(pages_of(n) for n in held)
    spare = sum(pages_of(k + n) for k, n in zip(keep, new)) + 7
    order = _perm(g, used + spare)
    table = torch.full((case["S"], max_pages), -1, dtype=torch.int32, device=_DEV)
    h = torch.tensor([pages_of(n) for n in held], device=_DEV)
    mine = torch.arange(max_pages, device=_DEV)[None, :] < h[:, None]
    table[mine] = order[:used]
    free = torch.full((used + spare,), -1, dtype=torch.int32, device=_DEV)
    free[:spare] = order[used:]
    return dict(case, held=_i32(held), keep=_i32(keep), new=_i32(new), table=table, free=free, count=_i32([spare]),
                pages=used + spare, tokens=sum(new) + 5)  # the last tokens of the step's batch are padding


def _prepare_rope(case, g):
    Hq, Hkv, D, rot = case["Hq"], case["Hkv"], case["D"], case["rot"]
    w = lambda: (1.0 + 0.3 * torch.randn(D, generator=g, device=_DEV)).bfloat16() if case["norm"] else None  # noqa: E731
    s = dict(case, q_weight=w(), k_weight=w())
    heads = Hq + 2 * Hkv
    if case["way"] == "append":
        N, page = case["N"], case["page"]
        pages = (N + page - 1) // page + 3
        s["cos"], s["sin"] = _table(32768, rot)
        s["positions"] = torch.randint(0, 32768, (N,), generator=g, device=_DEV, dtype=torch.int32)
        qkv = _normal(g, N, heads, D)  # the fused projection's output
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["slots"] = _slots(g, N, page, pages)
        s["k_pool"], s["v_pool"] = _normal(g, pages, page, Hkv, D), _normal(g, pages, page, Hkv, D)
        return s
    B, T = case["B"], case["T"]
    s["cos"], s["sin"] = _table(T, rot)
    s["positions"] = torch.arange(T, dtype=torch.int32, device=_DEV)
    qkv = _normal(g, B, T, heads, D).transpose(1, 2)  # [B, heads, T, D] as the projection leaves it
    s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    if case["way"] == "backward":
        s["dq"], s["dk"] = _normal(g, B, Hq, T, D), _normal(g, B, Hkv, T, D)
    return s


# ---------------------------------------------------------------- the plain forms
def _quantise(x):
    """Rows of bf16 values [..., D] as rows of the 4-bit cache [..., D/2 + 4] bytes."""
    x = x.float()
    m = x.amin(-1, keepdim=True)
    step = ((x.amax(-1, keepdim=True) - m) / 15).bfloat16()
    inv = torch.where(step > 0, 1 / step.float(), torch.zeros_like(m))
    code = ((x - m).double() * inv.double()).round().to(torch.uint8)  # 64 bits: values next to a border
    head = torch.cat([step, m.bfloat16()], -1).view(torch.uint8)
    return torch.cat([code[..., 0::2] | (code[..., 1::2] << 4), head], -1)


def _values(rows):
    """What rows of the 4-bit cache stand for, in 32 bits."""
    head = rows[..., -4:].contiguous().view(torch.bfloat16).float()
    code = torch.stack([rows[..., :-4] & 15, rows[..., :-4] >> 4], -1).flatten(-2)
    return code.float() * head[..., :1] + head[..., 1:]


def _rotate(x, cos, sin, rot, pairs):
    """Rotate the first `rot` elements of the last axis; cos, sin broadcast over [..., rot/2]."""
    r, rest = x[..., :rot], x[..., rot:]
    if pairs == "halves":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


_EPS = 1e-6


def _norm_rope(s, x, w, cos, sin):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * w.float()
    return _rotate(x, cos, sin, s["rot"], s["pairs"])


def _norm_rope_back(s, d, x, w, cos, sin):
    """(gradient of x in bf16, gradient of w in fp32 or None) for the output gradient d [B, H, T, D]."""
    d = _rotate(d.float(), cos, -sin, s["rot"], s["pairs"])
    if w is None:
        return d.bfloat16(), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS)
    n = x * r
    e = d * w.float()
    return (r * (e - n * (e * n).mean(-1, keepdim=True))).bfloat16(), (d * n).sum((0, 1, 2))


def _run_plan(s):
    page, held, keep, new, table, free = s["page"], s["held"].long(), s["keep"].long(), s["new"].long(), s["table"], s["free"]
    count = s["count"].long()
    after = keep + new
    had, has = (held + page - 1) // page, (after + page - 1) // page
    take, give = (has - had).clamp(min=0), (had - has).clamp(min=0)
    end_take, end_give = take.cumsum(0), give.cumsum(0)
    n_take, n_give = end_take[-1:], end_give[-1:]
    some = torch.arange(free.numel(), device=_DEV)
    # released pages, in the order in which they are pushed
    who = torch.searchsorted(end_give, some, right=True).clamp(max=held.numel() - 1)
    where = has[who] + some - (end_give - give)[who]
    pushed = table[who, where.clamp(0, table.shape[1] - 1)]
    # taken pages, in the order in which they are popped
    back = n_give - 1 - some
    popped = torch.where(back >= 0, pushed[back.clamp(min=0)], free[(count + back).clamp(0, free.numel() - 1)])
    stay = n_give - torch.minimum(n_give, n_take)
    at = torch.where(some < stay, count + some, free.numel())
    free_out = torch.cat([free, free[:1]]).scatter(0, at, pushed)[:-1]
    cols = torch.arange(table.shape[1], device=_DEV)[None, :]
    fresh = (cols >= had[:, None]) & (cols < has[:, None])
    n = ((end_take - take)[:, None] + cols - had[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, popped[n], table))
    free.copy_(free_out)
    end = new.cumsum(0)
    cu = torch.cat([torch.zeros_like(end[:1]), end])
    t = torch.arange(s["tokens"], device=_DEV)
    seq = torch.searchsorted(end, t, right=True)
    real = seq < held.numel()
    seq = seq.clamp(max=held.numel() - 1)
    pos = torch.where(real, keep[seq] + t - cu[seq], 0)
    slot = torch.where(real, table[seq, pos // page].long() * page + pos % page, -1)
    i = lambda x: x.to(torch.int32)  # noqa: E731
    return {"seqlens_k": i(after), "cu_seqlens": i(cu), "positions": i(pos), "slots": i(slot),
            "free_count": i(count + n_give - n_take), "table": table, "free": free}


def _run_decode(s):
    q, lens, page, Tq, Hkv, D = s["q"], s["lens"], s["page"], s["Tq"], s["Hkv"], s["D"]
    B, Hq = q.shape[:2]

    def rows(pool):  # [B, Hkv, keys, D] in 32 bits, padded to the longest
        return _values(pool[s["table"].long()].transpose(1, 2).flatten(2, 3))

    sc = q.float().reshape(B, Hkv, Hq // Hkv * Tq, D) @ rows(s["k_pool"]).transpose(2, 3)
    sc = (sc * D ** -0.5).view(B, Hkv, Hq // Hkv, Tq, -1)
    pos = lens[:, None].long() - Tq + torch.arange(Tq, device=_DEV)
    key = torch.arange(sc.shape[-1], device=_DEV)
    see = key <= pos[:, :, None]
    if s["window"]:
        see &= key > pos[:, :, None] - s["window"]
    see = see[:, None, None]
    sc = sc.masked_fill(~see, float("-inf"))
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top.isinf(), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)  # a row that sees no key gives zeros
    return (p.view(B, Hkv, -1, p.shape[-1]) @ rows(s["v_pool"])).view(B, Hq, Tq, D).bfloat16()


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "plan":
        return _run_plan(s)
    if s["op"] == "decode4":
        return _run_decode(s)
    if s["op"] == "kv4":
        page, at = s["page"], s["slots"].long()
        for pool, x in ((s["k_pool"], s["k"]), (s["v_pool"], s["v"])):
            pool[at // page, :, at % page] = _quantise(x)
        return {p: _values(s[p + "_pool"][at // page, :, at % page]).bfloat16() for p in ("k", "v")}
    cos, sin = s["cos"][s["positions"].long()], s["sin"][s["positions"].long()]
    if s["way"] == "append":
        cos, sin = cos[:, None], sin[:, None]
        page, at = s["page"], s["slots"].long()
        s["k_pool"][at // page, at % page] = _norm_rope(s, s["k"], s["k_weight"], cos, sin).bfloat16()
        s["v_pool"][at // page, at % page] = s["v"]
        return {"q": _norm_rope(s, s["q"], s["q_weight"], cos, sin).bfloat16(), "k_pool": s["k_pool"],
                "v_pool": s["v_pool"]}
    if s["way"] == "forward":
        return {"q": _norm_rope(s, s["q"], s["q_weight"], cos, sin).bfloat16(),
                "k": _norm_rope(s, s["k"], s["k_weight"], cos, sin).bfloat16()}
    dq, dq_weight = _norm_rope_back(s, s["dq"], s["q"], s["q_weight"], cos, sin)
    dk, dk_weight = _norm_rope_back(s, s["dk"], s["k"], s["k_weight"], cos, sin)
    return {"dq": dq, "dk": dk, "dq_weight": dq_weight, "dk_weight": dk_weight}


# ---------------------------------------------------------------- the library's calls
def _run_own(s):
    import grouped_query_softmax_b200 as gqa
    if s["op"] == "plan":
        p = gqa.paged_plan(s["held"], s["new"], s["table"], s["free"], s["count"], page_size=s["page"],
                           num_pages=s["pages"], max_tokens=s["tokens"], keep=s["keep"])
        return {"seqlens_k": p.seqlens_k, "cu_seqlens": p.cu_seqlens, "positions": p.positions, "slots": p.slots,
                "free_count": p.free_count, "table": s["table"], "free": s["free"]}
    if s["op"] == "decode4":
        return gqa.attn_decode_kv4(s["q"], s["k_pool"], s["v_pool"], s["lens"], s["table"], max_seqlen_k=s["longest"],
                                   window=s["window"])
    if s["op"] == "kv4":
        gqa.kv4_append(s["k"], s["v"], s["k_pool"], s["v_pool"], s["slots"])
        k, v = gqa.kv4_gather(s["k_pool"], s["v_pool"], s["slots"])
        return {"k": k, "v": v}
    how = {"q_weight": s["q_weight"], "k_weight": s["k_weight"], "eps": _EPS, "cos": s["cos"], "sin": s["sin"],
           "positions": s["positions"], "interleaved": s["pairs"] == "neighbours"}
    if s["way"] == "append":
        q = gqa.qk_norm_rope_append(s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["slots"], **how)
        return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if s["way"] == "forward":
        q, k = gqa.qk_norm_rope(s["q"], s["k"], **how)
        return {"q": q, "k": k}
    dq, dk, dq_weight, dk_weight = gqa.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], **how)
    return {"dq": dq, "dk": dk, "dq_weight": dq_weight, "dk_weight": dk_weight}


# ---------------------------------------------------------------- work and the definition in 64 bits
def work(case):
    if case["op"] == "plan":
        held, keep, new = _plan_lengths(case)
        page, S, N = case["page"], case["S"], sum(new) + 5
        moved = sum(abs((k + n + page - 1) // page - (h + page - 1) // page) for h, k, n in zip(held, keep, new))
        # three lengths in, two out, a page number moved once in and once out, two values a token
        return {"bytes": 4 * (5 * S + 3 + 2 * moved + 2 * N), "flops": 0}
    if case["op"] == "decode4":
        lens, Tq, w = _decode_lengths(case), case["Tq"], case["window"]
        keys = sum(n - (max(0, n - Tq - w + 1) if w else 0) for n in lens)
        pairs = sum(max(0, min(p + 1, w) if w else p + 1) for n in lens for p in range(n - Tq, n))
        rows = case["B"] * case["Hq"] * Tq * case["D"] * 2
        return {"bytes": keys * case["Hkv"] * 2 * (case["D"] // 2 + 4) + 2 * rows + 4 * (case["B"] + keys // case["page"]),
                "flops": 4 * case["D"] * case["Hq"] * pairs}
    if case["op"] == "kv4":
        row = case["N"] * case["Hkv"] * 2
        # bf16 in, 4 bits out, and the other way
        return {"bytes": row * 2 * (2 * case["D"] + case["D"] // 2 + 4) + 8 * case["N"], "flops": 0}
    tokens = case["N"] if case["way"] == "append" else case["B"] * case["T"]
    heads = case["Hq"] + case["Hkv"]
    unit = tokens * case["D"] * 2
    angles = (32768 if tokens > 32768 else tokens) if case["way"] == "append" else case["T"]
    small = angles * case["rot"] * 4 + 4 * tokens
    if case["way"] == "append":
        return {"bytes": 2 * unit * (heads + case["Hkv"]) + small + 4 * tokens, "flops": 0}
    moved = 2 if case["way"] == "forward" or not case["norm"] else 3
    return {"bytes": moved * unit * heads + small, "flops": 0}


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "kv4":
        out = {}
        for p in ("k", "v"):
            x = s[p].to(f8)
            low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            step = ((high - low) / 15).float().bfloat16().to(f8)
            scale = (1.0 / step.float()).to(f8)  # the definition rounds it to 32 bits: ties go by it
            code = torch.where(step > 0, torch.round((x - low) * scale), torch.zeros_like(x))
            out[p] = low + step * code
        return out
    if case["op"] == "decode4":
        return _exact_decode(s)

    def turn(x, sign):  # rotation by sign * angle as a product of complex numbers
        R, H = case["rot"], case["rot"] // 2
        at = s["positions"].long()
        z = torch.complex(s["cos"].to(f8)[at], sign * s["sin"].to(f8)[at])
        z = z[:, None] if case["way"] == "append" else z
        i = torch.arange(H, device=x.device)
        first, second = (i, i + H) if case["pairs"] == "halves" else (2 * i, 2 * i + 1)
        y = torch.complex(x[..., first], x[..., second]) * z
        out = x.clone()
        out[..., first], out[..., second] = y.real, y.imag
        return out

    def normed(x, w):
        if w is None:
            return x.to(f8), None, None
        x = x.to(f8)
        size = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + _EPS).sqrt()
        return x / size * w.to(f8), x / size, size

    if case["way"] == "append":
        k = turn(normed(s["k"], s["k_weight"])[0], 1.0)
        pools = {}
        for name, x in (("k_pool", k), ("v_pool", s["v"].to(f8))):
            flat = s[name].to(f8).flatten(0, 1).clone()
            flat[s["slots"].long()] = x
            pools[name] = flat.view(s[name].shape)
        return dict(pools, q=turn(normed(s["q"], s["q_weight"])[0], 1.0))
    if case["way"] == "forward":
        return {"q": turn(normed(s["q"], s["q_weight"])[0], 1.0), "k": turn(normed(s["k"], s["k_weight"])[0], 1.0)}
    out = {}
    for p in ("q", "k"):
        d = turn(s["d" + p].to(f8), -1.0)
        w = s[p + "_weight"]
        _, unit, size = normed(s[p], w)
        out["d%s_weight" % p] = None
        if w is not None:
            out["d%s_weight" % p] = torch.einsum("bhtd,bhtd->d", d, unit)
            d = d * w.to(f8)
            d = (d - unit * torch.einsum("bhtd,bhtd->bht", d, unit)[..., None] / d.shape[-1]) / size
        out["d" + p] = d
    return out


def _exact_decode(s):
    q, page, Tq, D = s["q"].to(torch.float64), s["page"], s["Tq"], s["D"]
    out = torch.zeros_like(q)
    G = s["Hq"] // s["Hkv"]
    for b, n in enumerate(_decode_lengths({k: s[k] for k in s if not isinstance(s[k], torch.Tensor) and k != "longest"})):
        t = torch.arange(n, device=q.device)
        at = s["table"][b].long()[t // page]

        def rows(pool):
            r = pool[at, :, t % page]  # [n, Hkv, bytes]
            head = r[..., D // 2:].contiguous().view(torch.bfloat16).to(torch.float64)
            x = torch.empty(n, s["Hkv"], D, dtype=torch.float64, device=q.device)
            x[..., 0::2], x[..., 1::2] = (r[..., :D // 2] % 16).to(torch.float64), (r[..., :D // 2] // 16).to(torch.float64)
            return x.mul_(head[..., :1]).add_(head[..., 1:])

        pos = n - Tq + torch.arange(Tq, device=q.device)
        see = t[None] <= pos[:, None]
        if s["window"]:
            see &= t[None] > pos[:, None] - s["window"]
        sc = torch.einsum("kgid,tkd->kgit", q[b].view(s["Hkv"], G, Tq, D), rows(s["k_pool"])) / D ** 0.5
        p = sc.masked_fill(~see, float("-inf")).softmax(-1).nan_to_num(0.0)
        out[b] = torch.einsum("kgit,tkd->kgid", p, rows(s["v_pool"])).reshape(s["Hq"], Tq, D)
    return out
