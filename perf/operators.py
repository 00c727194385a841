"""Cases of the serving-step operators: block tables, query / key norm with
rotation and cache write, attention over the 8-bit paged cache, and the
verification of drafted tokens.

``run(state)`` is one pass through one operator.  With ``own`` false it is
the operator's plain form in elementary torch operations; with ``own`` true
it is the framework's call on the same inputs.  ``exact`` evaluates the
definition in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

D = 128              # head dimension
E4M3_MAX = 448.0     # largest e4m3 value
EXP_MIN, EXP_MAX = -64, 119   # range of the page scales' exponents
DEV = "cuda"


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a small batch, and a mixed batch of long prompts and decodes
        dict(name="tables_n64", op="tables", B=64, new_max=1, ctx_max=8192, bs=64, pad=0),
        dict(name="tables_mixed", op="tables", B=1024, new_max=300, ctx_max=20000, bs=16, pad=1001),
        # the smallest decode batch; a speculative batch of 64 sequences x 4 tokens; a prompt batch of 16,384 tokens
        dict(name="rope_n4", op="rope", B=4, new=1, Hq=12, Hkv=4, bs=16, rot=128, inter=False, ctx_max=700, pad=0),
        dict(name="rope_spec", op="rope", B=64, new=4, Hq=48, Hkv=8, bs=64, rot=64, inter=True, ctx_max=100000, pad=5),
        dict(name="rope_prompt", op="rope", B=16, new=1024, Hq=48, Hkv=8, bs=64, rot=128, inter=False, ctx_max=900,
             pad=0),
        # the smallest decode batch with short contexts; a speculative batch over ragged contexts; one sequence with
        # a very long context; prompt chunks attending to what is cached
        dict(name="attn_n4", op="attn", B=4, new=1, Hq=12, Hkv=4, bs=16, len_min=1, len_max=700, ragged=False),
        dict(name="attn_spec", op="attn", B=64, new=4, Hq=48, Hkv=8, bs=64, len_min=1000, len_max=16384, ragged=False),
        dict(name="attn_long", op="attn", B=1, new=1, Hq=96, Hkv=8, bs=128, len_min=260001, len_max=260001,
             ragged=False),
        dict(name="attn_prompt", op="attn", B=4, new=515, Hq=48, Hkv=8, bs=32, len_min=600, len_max=4100, ragged=True),
        # one sequence; a batch of drafts without draft probabilities and an odd vocabulary; a large batch
        dict(name="verify_n1", op="verify", B=1, T=4, V=131072, probs=True),
        dict(name="verify_odd", op="verify", B=33, T=8, V=100003, probs=False),
        dict(name="verify_n256", op="verify", B=256, T=4, V=131072, probs=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "attn", "verify"])
    heads = rng.choice([(12, 4), (12, 12), (48, 8), (96, 8), (40, 8), (16, 1), (7, 7), (33, 11)])
    bs = rng.choice([16, 32, 64, 128])
    if op == "tables":
        return dict(op=op, B=_log(rng, 1, 1500), new_max=rng.choice([1, 4, 60, 300]), ctx_max=_log(rng, 100, 20000),
                    bs=bs, pad=rng.choice([0, rng.randrange(2000)]))
    if op == "rope":
        new = rng.choice([1, rng.randrange(2, 9), _log(rng, 9, 500)])
        Hq, Hkv = heads if heads[0] <= 48 else (48, 8)
        return dict(op=op, B=_log(rng, 1, min(256, 12000 // new)), new=new, Hq=Hq, Hkv=Hkv, bs=bs,
                    rot=rng.choice([128, 64, 32, 0]), inter=rng.random() < 0.5, ctx_max=_log(rng, 100, 1000000),
                    pad=rng.choice([0, rng.randrange(40)]))
    if op == "attn":
        if rng.random() < 0.25:
            return dict(op=op, B=rng.randrange(1, 5 if heads[0] <= 48 else 3), new=_log(rng, 9, 500), Hq=heads[0],
                        Hkv=heads[1], bs=bs, len_min=600, len_max=_log(rng, 700, 4100), ragged=True)
        B = _log(rng, 1, 128)
        hi = _log(rng, 30, max(200, min(100000, 500000 // (B * (heads[1] // 8 + 1)))))
        return dict(op=op, B=B, new=rng.choice([1, 1, rng.randrange(2, 9)]), Hq=heads[0], Hkv=heads[1], bs=bs,
                    len_min=rng.choice([1, hi // 2 + 1]), len_max=hi, ragged=rng.random() < 0.3)
    return dict(op=op, B=_log(rng, 1, 256), T=rng.randrange(1, 9), V=_log(rng, 300, 131072),
                probs=rng.random() < 0.6)


# -------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(v, dt=torch.int32):
    return torch.tensor(v, dtype=dt, device=DEV)


def _lens(case, seed=None):
    """cached and new tokens of each request, host lists.  A case has the same requests for every seed, in an order
    of the seed's: tensors keep their sizes from one batch to the next, as in a program that captures its step."""
    rng = random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))
    B = case["B"]
    if case["op"] == "tables":
        new = [rng.randint(0 if case["new_max"] > 1 else 1, case["new_max"]) if rng.random() < 0.3 else 1
               for _ in range(B)]
        ctx = [rng.randint(0, case["ctx_max"]) for _ in range(B)]
    elif case["op"] == "rope":
        ctx, new = [rng.randint(0, case["ctx_max"]) for _ in range(B)], [case["new"]] * B
    else:
        new = [rng.randint(1, case["new"]) if case["ragged"] else case["new"] for _ in range(B)]
        if case["ragged"]:
            new[0] = case["new"]
        lo, hi = case["len_min"], case["len_max"]
        ctx = [max(n, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) if lo < hi else hi) - n for n in new]
    both = list(zip(ctx, new))
    if seed is not None:
        random.Random(seed).shuffle(both)
    return [c for c, _ in both], [n for _, n in both]


def _cu(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cu


def _e4m3(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float16).mul_(60).clamp_(-440, 440).to(
        torch.float8_e4m3fn)


def _scales(shape, g):
    # page scales are powers of two; the rows of a page then have about unit size
    return torch.exp2(torch.randint(-7, -4, shape, generator=g, device=DEV).float())


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case, op=case["op"])
    if case["op"] == "verify":
        B, T, V = case["B"], case["T"], case["V"]
        # target rows and, near them, the draft model's rows; drafted tokens follow the draft's probabilities
        logit = torch.randn(B, T, V, generator=g, device=DEV) * 3
        s["target_probs"] = torch.softmax(logit, -1)
        near = torch.softmax(logit[:, :T - 1] + 0.6 * torch.randn(B, T - 1, V, generator=g, device=DEV), -1)
        r = torch.rand(B, max(T - 1, 0), 1, generator=g, device=DEV)
        s["draft_tokens"] = (near.cumsum(-1) < r).sum(-1).clamp_(max=V - 1).int()
        s["draft_probs"] = near.contiguous() if case["probs"] else None
        s["accept_u"] = torch.rand(B, max(T - 1, 0), generator=g, device=DEV)
        s["sample_u"] = torch.rand(B, generator=g, device=DEV)
        s["slots"] = (torch.randperm(B * T, generator=g, device=DEV) + 1).int().view(B, T)
        del logit
        if own:
            from linear_attention_decode_04_gb300 import KdaVerifyDraftCall
            s["call"] = KdaVerifyDraftCall(s["draft_tokens"], s["target_probs"], s["accept_u"], s["sample_u"],
                                           draft_probs=s["draft_probs"], slot_idx=s["slots"])
        return s
    ctx, new = _lens(case, seed)
    B, bs = case["B"], case["bs"]
    cu = _cu(new)
    T = cu[-1] + case.get("pad", 0)
    pages = [-(-(c + n) // bs) for c, n in zip(ctx, new)]
    if case["op"] == "tables":
        M, total = max(pages) + 3, sum(pages)
        ids = torch.randperm(total + 64, generator=g, device=DEV).int()
        table = torch.full((B, M), -1, dtype=torch.int32, device=DEV)
        held = torch.arange(M, device=DEV) < _ints([-(-c // bs) for c in ctx])[:, None]
        rank = held.view(-1).cumsum(0).view(B, M) - 1
        table = torch.where(held, ids[rank.clamp(min=0)], table)
        used = int(held.sum())
        s.update(cached_lens=_ints(ctx), new_lens=_ints(new), block_table=table,
                 free_blocks=torch.cat([ids[:5], ids[used:]]).contiguous(), free_head=_ints([5]), T=T)
        if own:
            from linear_attention_decode_04_gb300 import KdaBlockTablesCall
            s["call"] = KdaBlockTablesCall(s["cached_lens"], s["new_lens"], table, s["free_blocks"], s["free_head"],
                                           block_size=bs, num_blocks=total + 64, num_tokens=T)
        return s
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "rope":
        # the cache holds the pages that this step writes (and a few more): the context's other pages are not met
        pos, slot, at = [], [], 0
        for c, n in zip(ctx, new):
            pos += range(c, c + n)
            slot += [at * bs + c % bs + j for j in range(n)]
            at += -(-(c % bs + n) // bs)
        nb = at + 3
        perm = torch.randperm(nb - 1, generator=g, device=DEV)
        slot = _ints(slot, torch.int64)
        slot = perm[slot // bs] * bs + slot % bs
        pad = T - cu[-1]
        s.update(qkv=torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=DEV).bfloat16(),
                 positions=torch.cat([_ints(pos), torch.zeros(pad, dtype=torch.int32, device=DEV)]),
                 slot_map=torch.cat([slot, torch.full((pad,), -1, dtype=torch.int64, device=DEV)]),
                 q_weight=1 + 0.1 * torch.randn(D, generator=g, device=DEV),
                 k_weight=1 + 0.1 * torch.randn(D, generator=g, device=DEV),
                 k_cache=_e4m3((nb, Hkv, bs, D), g), v_cache=_e4m3((nb, Hkv, bs, D), g),
                 k_scale=_scales((nb, Hkv), g), v_scale=_scales((nb, Hkv), g),
                 q_out=torch.zeros(T, Hq * D, dtype=torch.bfloat16, device=DEV), base=1e6)
        if own:
            from linear_attention_decode_04_gb300 import KdaQkRopeCall, rope_frequencies
            s["call"] = KdaQkRopeCall(s["qkv"], s["positions"], s["q_out"], num_q_heads=Hq, num_kv_heads=Hkv,
                                      rope_freqs=rope_frequencies(case["rot"], s["base"], device=DEV),
                                      interleaved=case["inter"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                      eps=1e-6, k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"],
                                      v_scale=s["v_scale"], slot_map=s["slot_map"])
        return s
    M, nb = max(pages), sum(pages) + 3
    ids = torch.randperm(nb, generator=g, device=DEV).int()
    table = torch.full((B, M), -1, dtype=torch.int32, device=DEV)
    row = torch.repeat_interleave(torch.arange(B, device=DEV), _ints(pages, torch.int64))
    first = _ints(_cu(pages)[:-1], torch.int64)
    table[row, torch.arange(row.numel(), device=DEV) - first[row]] = ids[:row.numel()]
    s.update(q=torch.randn(T, Hq * D, generator=g, device=DEV).bfloat16(), cu_seqlens=_ints(cu),
             seq_lens=_ints([c + n for c, n in zip(ctx, new)]), block_table=table,
             k_cache=_e4m3((nb, Hkv, bs, D), g), v_cache=_e4m3((nb, Hkv, bs, D), g),
             k_scale=_scales((nb, Hkv), g), v_scale=_scales((nb, Hkv), g),
             out=torch.zeros(T, Hq * D, dtype=torch.bfloat16, device=DEV), max_new=max(new), max_len=M * bs,
             host=(cu, [c + n for c, n in zip(ctx, new)]))
    if own:
        from linear_attention_decode_04_gb300 import KdaCacheAttentionCall
        s["call"] = KdaCacheAttentionCall(s["q"], s["cu_seqlens"], s["seq_lens"], table, s["k_cache"], s["v_cache"],
                                          s["k_scale"], s["v_scale"], s["out"], max_new=s["max_new"])
    return s


# ---------------------------------------------------------------------- run
def run(s):
    if own:
        return _run_own(s)
    return dict(tables=_tables, rope=_rope, attn=_attn, verify=_verify)[s["op"]](s)


def _run_own(s):
    c = s["call"]
    c()
    if s["op"] == "tables":
        return dict(block_table=s["block_table"], cu_seqlens=c.cu_seqlens, seq_lens=c.seq_lens,
                    positions=c.positions, slot_map=c.slot_map, free_head=c.free_head_out)
    if s["op"] == "rope":
        return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"],
                    v_scale=s["v_scale"])
    if s["op"] == "attn":
        return dict(out=s["out"])
    return dict(tokens=c.tokens, num_accepted=c.num_accepted, next_slot=c.next_slot)


def _tables(s):
    c, n, bs, T = s["cached_lens"].long(), s["new_lens"].long(), s["case"]["bs"], s["T"]
    table, free = s["block_table"], s["free_blocks"].long()
    B, M = table.shape
    end = n.cumsum(0)
    start = end - n
    first, need = (c + bs - 1) // bs, (c + n + bs - 1) // bs - (c + bs - 1) // bs
    off = s["free_head"].long() + need.cumsum(0) - need
    t = torch.arange(T, device=DEV)
    i = torch.searchsorted(end, t, right=True)
    valid = i < B
    i = i.clamp(max=B - 1)
    pos = c[i] + t - start[i]
    page = torch.where(valid, pos // bs, 0)
    fresh = valid & (page >= first[i])
    blk = torch.where(fresh, free[torch.where(fresh, off[i] + page - first[i], 0)], table[i, page].long())
    opens = fresh & (pos % bs == 0)
    flat = torch.cat([table.view(-1), table.new_zeros(1)])
    flat[torch.where(opens, i * M + page, B * M)] = blk.int()
    table.copy_(flat[:-1].view(B, M))
    return dict(block_table=table, cu_seqlens=torch.cat([end.new_zeros(1), end]).int(), seq_lens=(c + n).int(),
                positions=torch.where(valid, pos, 0).int(), slot_map=torch.where(valid, blk * bs + pos % bs, -1),
                free_head=(s["free_head"] + need.sum()).int())


def _inv_freq(rot, base):
    return torch.pow(torch.tensor(base, dtype=torch.float64, device=DEV),
                     -torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)


def _norm_rotate(x, w, cos, sin, inter):
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    r = 2 * cos.shape[-1]
    h, rest = x[..., :r], x[..., r:]
    a, b = (h[..., 0::2], h[..., 1::2]) if inter else (h[..., :r // 2], h[..., r // 2:])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([ya, yb], -1).flatten(-2) if inter else torch.cat([ya, yb], -1)
    return torch.cat([y, rest], -1)


def _page_scale(amax):
    m, e = torch.frexp(amax)   # amax = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), EXP_MIN).clamp(EXP_MIN, EXP_MAX)
    return torch.exp2(e.float())


def _store(cache, scale, x, page, off, valid):
    """x [T, Hkv, D] into pages: the page's scale grows to what the new rows need, older rows follow it"""
    nb, Hkv, bs, _ = cache.shape
    amax = scale.new_zeros(nb, Hkv).scatter_reduce_(
        0, page[:, None].expand(-1, Hkv), torch.where(valid[:, None], x.abs().amax(-1), 0), "amax")
    first = torch.full((nb,), bs, dtype=torch.int64, device=DEV).scatter_reduce_(
        0, page, torch.where(valid, off, bs), "amin")
    fit = _page_scale(amax)
    new = torch.where((first < bs)[:, None], torch.where((first > 0)[:, None], torch.maximum(scale, fit), fit), scale)
    older = (torch.arange(bs, device=DEV) < first[:, None]) & (first < bs)[:, None]
    ratio = torch.where(older[:, None, :], (scale / new)[:, :, None], 1.0)
    full = (cache.float() * ratio[..., None]).to(torch.float8_e4m3fn)
    code = (x / new[page][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    keep = full[nb - 1, :, 0].view(torch.uint8)   # padding rows put back what a page outside every table holds
    full.view(torch.uint8)[page, :, off] = torch.where(valid[:, None, None], code.view(torch.uint8), keep)
    cache.copy_(full)
    scale.copy_(new)


def _rope(s):
    case = s["case"]
    Hq, Hkv, bs, nb = case["Hq"], case["Hkv"], case["bs"], s["k_cache"].shape[0]
    x = s["qkv"].float().view(-1, Hq + 2 * Hkv, D)
    ang = s["positions"].double()[:, None] * _inv_freq(case["rot"], s["base"])
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    q = _norm_rotate(x[:, :Hq], s["q_weight"], cos, sin, case["inter"])
    k = _norm_rotate(x[:, Hq:Hq + Hkv], s["k_weight"], cos, sin, case["inter"])
    valid = s["slot_map"] >= 0
    page, off = torch.where(valid, s["slot_map"] // bs, nb - 1), torch.where(valid, s["slot_map"] % bs, 0)
    _store(s["k_cache"], s["k_scale"], k, page, off, valid)
    _store(s["v_cache"], s["v_scale"], x[:, Hq + Hkv:], page, off, valid)
    s["q_out"].copy_(q.reshape(q.shape[0], -1))
    return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _attn(s):
    case, cu, lens = s["case"], s["cu_seqlens"].long(), s["seq_lens"].long()
    Hq, Hkv, n = case["Hq"], case["Hkv"], s["max_new"]
    G, B, L = Hq // Hkv, case["B"], s["max_len"]
    page = s["block_table"].long().clamp(min=0)

    def rows(cache, scale):   # [B, Hkv, L, D]
        x = cache[page].float() * scale[page][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, L, D)

    count = cu[1:] - cu[:-1]
    j = torch.arange(n, device=DEV)
    T = s["q"].shape[0]
    q = s["q"][(cu[:-1, None] + j).clamp(max=T - 1)].float()
    q = q.view(B, n, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, n * G, D)
    z = (q @ rows(s["k_cache"], s["k_scale"]).transpose(-1, -2)).mul_(D ** -0.5)
    limit = (lens - count)[:, None] + j + 1                        # keys that query j of a sequence sees
    seen = torch.arange(L, device=DEV) < limit[:, :, None]
    z.view(B, Hkv, n, G, L).masked_fill_(~seen[:, None, :, None], float("-inf"))
    z = z.sub_(z.amax(-1, keepdim=True)).exp_()
    o = (z @ rows(s["v_cache"], s["v_scale"])) / z.sum(-1, keepdim=True)
    o = o.view(B, Hkv, n, G, D).transpose(1, 2).reshape(B, n, Hq * D)
    t = torch.arange(T, device=DEV)
    i = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    s["out"].copy_(o[i, t - cu[i]])
    return dict(out=s["out"])


def _verify(s):
    p, u = s["target_probs"], s["accept_u"]
    B, T, V = p.shape
    d = s["draft_tokens"].long()
    pd = p[:, :T - 1].gather(-1, d[..., None])[..., 0].double()
    if s["draft_probs"] is not None:
        qd = s["draft_probs"].gather(-1, d[..., None])[..., 0].double()
    else:
        qd = torch.ones_like(pd)
    ok = (u.double() * qd < pd).long().cumprod(-1)
    k = ok.sum(-1)                                              # drafts accepted
    b = torch.arange(B, device=DEV)

    def fixed(x):                                               # probabilities in units of 2^-60
        return (x.clamp(0, 1) * 2.0 ** 60).long()

    w = fixed(p[b, k])
    if T > 1:
        last = (k == T - 1)[:, None]
        at = k.clamp(max=T - 2)
        if s["draft_probs"] is not None:
            q = fixed(s["draft_probs"][b, at])
        else:
            q = torch.where(torch.arange(V, device=DEV) == d[b, at][:, None], w, 0)
        rest = torch.where(last, w, (w - q).clamp(min=0))
        w = torch.where((rest.sum(-1) > 0)[:, None], rest, w)
    cum = w.cumsum(-1)
    total = cum[:, -1]
    r = (s["sample_u"].double() * 2.0 ** 31).long()
    target = r * (total >> 31) + ((r * (total & (2 ** 31 - 1))) >> 31)
    x = (cum <= target[:, None]).sum(-1)
    j = torch.arange(T, device=DEV)
    tok = torch.cat([d, d.new_full((B, 1), -1)], 1)
    tok = torch.where(j < k[:, None], tok, torch.where(j == k[:, None], x[:, None], -1))
    return dict(tokens=tok.int(), num_accepted=k.int(), next_slot=s["slots"][b, k])


# --------------------------------------------------------------------- work
def work(case):
    if case["op"] == "verify":
        rows = 2 if case["probs"] else 1
        n = case["B"] * case["T"]
        return {"bytes": case["B"] * case["V"] * 4.0 * rows + 20.0 * n, "flops": 3.0 * case["B"] * case["V"]}
    ctx, new = _lens(case)
    T, B, bs = sum(new), case["B"], case["bs"]
    if case["op"] == "tables":
        fresh = sum(-(-(c + n) // bs) - -(-c // bs) for c, n in zip(ctx, new))
        return {"bytes": 12.0 * (T + case["pad"]) + 20.0 * B + 8.0 * fresh, "flops": 10.0 * T}
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "rope":
        # rows in, queries and cache rows out, and the scales
        return {"bytes": T * ((Hq + 2 * Hkv) * 2.0 * D + Hq * 2.0 * D + 2.0 * Hkv * D + 12), "flops":
                T * (10.0 * (Hq + Hkv) + 3.0 * Hkv) * D}
    seen = sum(n * (c + c + n + 1) / 2 for c, n in zip(ctx, new))
    return {"bytes": sum(c + n for c, n in zip(ctx, new)) * 2.0 * Hkv * D + T * Hq * 4.0 * D,
            "flops": 4.0 * seen * Hq * D}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    s = _inputs(case, seed)
    return dict(tables=_exact_tables, rope=_exact_rope, attn=_exact_attn, verify=_exact_verify)[case["op"]](case, s)


def _inputs(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _exact_tables(case, s):
    bs, table, free = case["bs"], s["block_table"].tolist(), s["free_blocks"].tolist()
    head, cu, lens, pos, slot = s["free_head"].item(), [0], [], [], []
    for i, (c, n) in enumerate(zip(s["cached_lens"].tolist(), s["new_lens"].tolist())):
        for p in range(-(-c // bs), -(-(c + n) // bs)):
            table[i][p] = free[head]
            head += 1
        cu.append(cu[-1] + n)
        lens.append(c + n)
        pos += range(c, c + n)
        slot += [table[i][q // bs] * bs + q % bs for q in range(c, c + n)]
    pad = s["T"] - len(pos)
    return dict(block_table=_ints(table), cu_seqlens=_ints(cu), seq_lens=_ints(lens), positions=_ints(pos + [0] * pad),
                slot_map=_ints(slot + [-1] * pad, torch.int64), free_head=_ints([head]))


def _exact_rope(case, s):
    Hq, Hkv, bs, rot, T = case["Hq"], case["Hkv"], case["bs"], case["rot"], s["qkv"].shape[0]
    x = s["qkv"].double().view(T, -1, D)
    i = torch.arange(rot // 2, device=DEV)
    ang = s["positions"].double()[:, None] * torch.exp(i.double() * (-2.0 / max(rot, 1) * math.log(s["base"])))
    turn = torch.polar(torch.ones_like(ang), ang)[:, None]      # each pair as a complex number
    at = (2 * i, 2 * i + 1) if case["inter"] else (i, i + rot // 2)

    def rotated(y, w):
        y = y / (y.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        z = torch.complex(y[..., at[0]], y[..., at[1]]) * turn
        y[..., at[0]], y[..., at[1]] = z.real, z.imag
        return y

    res = dict(q=rotated(x[:, :Hq].clone(), s["q_weight"]).reshape(T, -1))
    live = s["slot_map"] >= 0
    slot = s["slot_map"][live]
    page, off = slot // bs, slot % bs
    for name, y in (("k", rotated(x[:, Hq:Hq + Hkv].clone(), s["k_weight"])), ("v", x[:, Hq + Hkv:])):
        cache, scale, y = s[name + "_cache"].double(), s[name + "_scale"].double(), y[live]
        top = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand(-1, Hkv), y.abs().amax(-1), "amax")
        lowest = torch.full((len(scale),), bs, dtype=torch.int64, device=DEV).scatter_reduce_(0, page, off, "amin")
        met, opened = lowest < bs, lowest == 0
        e = torch.ceil(torch.log2(top.clamp(min=1e-300) / E4M3_MAX)).clamp(EXP_MIN, EXP_MAX)
        fit = torch.pow(2.0, e)
        new = torch.where(met[:, None], torch.where(opened[:, None], fit, torch.maximum(fit, scale)), scale)
        old = met[:, None] & (torch.arange(bs, device=DEV) < lowest[:, None])
        moved = (cache * (scale / new)[:, :, None, None]).float().to(torch.float8_e4m3fn).double()
        cache = torch.where(old[:, None, :, None], moved, cache)
        code = (y / new[page][..., None]).clamp(-E4M3_MAX, E4M3_MAX)
        step = torch.exp2(torch.floor(torch.log2(code.abs().clamp(min=2.0 ** -6))) - 3)
        cache[page, :, off] = torch.round(code / step) * step     # e4m3, ties to even
        res[name + "_cache"], res[name + "_scale"] = cache, new
    return res


def _exact_attn(case, s):
    Hq, Hkv, bs = case["Hq"], case["Hkv"], case["bs"]
    cu, lens = s["host"]
    out = torch.zeros(s["q"].shape[0], Hq, D, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        ids = s["block_table"][b, :-(-n // bs)].long()
        k, v = ((s[c + "_cache"][ids].double() * s[c + "_scale"][ids].double()[..., None, None]).permute(1, 0, 2, 3)
                .reshape(Hkv, -1, D)[:, :n] for c in "kv")
        m = cu[b + 1] - cu[b]
        q = s["q"][cu[b]:cu[b + 1]].double().view(m, Hkv, Hq // Hkv, D)
        z = torch.einsum("mhgd,hld->hgml", q, k) / math.sqrt(D)
        z += torch.full((m, n), float("-inf"), dtype=torch.float64, device=DEV).triu(n - m + 1)
        out[cu[b]:cu[b + 1]] = torch.einsum("hgml,hld->mhgd", torch.softmax(z, -1), v).reshape(m, Hq, D)
    return dict(out=out.view(-1, Hq * D))


def _exact_verify(case, s):
    d, B, T = s["draft_tokens"].tolist(), case["B"], case["T"]
    u, tokens, accepted = s["accept_u"].tolist(), [], []
    for b in range(B):
        p, k, w = s["target_probs"][b].double(), 0, None
        while k < T - 1:
            q = s["draft_probs"][b, k].double() if case["probs"] else \
                torch.nn.functional.one_hot(s["draft_tokens"][b, k].long(), case["V"]).double()
            if not u[b][k] * q[d[b][k]].item() < p[k][d[b][k]].item():
                w = (p[k] - q).clamp(min=0)
                break
            k += 1
        w = p[k] if w is None or w.sum().item() == 0 else w
        c = w.cumsum(0)
        x = torch.searchsorted(c, s["sample_u"][b:b + 1].double() * c[-1], right=True).item()
        tokens.append(d[b][:k] + [x] + [-1] * (T - 1 - k))
        accepted.append(k)
    k = _ints(accepted, torch.int64)
    return dict(tokens=_ints(tokens), num_accepted=k.int(), next_slot=s["slots"].gather(1, k[:, None])[:, 0])
