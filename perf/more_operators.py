"""Cases of the operators between and behind a serving step's layers: the
residual's addition with root-mean-square norm and 8-bit output, matrix
products with bias, activation and residual in their epilogue, and log
probabilities of given tokens with entropy and top alternatives.

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

E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100    # least largest value of a row that its scale is made for
EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # the norm in front of a projection: the smallest decode batch; a speculative batch of 64 sequences x 4 tokens
        # whose norm feeds an 8-bit product and, in bf16, something else; a prompt batch of 16,384 tokens
        dict(name="norm_n4", op="norm", T=4, D=2048, residual=True, norm=True, outs="q", pad=0),
        dict(name="norm_step", op="norm", T=256, D=6144, residual=True, norm=True, outs="both", pad=0),
        dict(name="norm_prompt", op="norm", T=16384, D=6144, residual=True, norm=True, outs="q", pad=0),
        # a layer's output rows (already normalised per head), columns of wider rows, made 8-bit for the product behind
        dict(name="quantise_rows", op="norm", T=2061, D=4608, residual=False, norm=False, outs="q", pad=1536),
        # projections into a layer's q, k, v channels: 12 heads for 4 sequences; 48 heads for 64 sequences x 4 tokens;
        # 48 heads for a prompt batch
        dict(name="linear_n4", op="linear", M=4, N=4608, K=2048, bits=8, act=None, bias=False, residual=False,
             out="bf16"),
        dict(name="linear_step", op="linear", M=256, N=18432, K=6144, bits=8, act=None, bias=False, residual=False,
             out="bf16"),
        dict(name="linear_prompt", op="linear", M=16384, N=18432, K=6144, bits=8, act=None, bias=False,
             residual=False, out="bf16"),
        # the gated half of a feed-forward block for 64 sequences; a ragged prompt batch with everything in the epilogue
        dict(name="linear_gated", op="linear", M=64, N=16384, K=6144, bits=16, act="silu_gated", bias=False,
             residual=False, out="bf16"),
        dict(name="linear_ragged", op="linear", M=2061, N=6001, K=4616, bits=16, act="gelu", bias=True, residual=True,
             out="bf16"),
        # one sequence's row; a speculative batch's rows, those behind the accepted tokens not asked for; the rows of
        # a prompt whose tokens are given, in bf16
        dict(name="logprobs_n1", op="logprobs", B=1, T=1, V=131072, top=5, bits=32, ragged=False),
        dict(name="logprobs_step", op="logprobs", B=64, T=4, V=131072, top=20, bits=32, ragged=True),
        dict(name="logprobs_prompt", op="logprobs", B=1, T=4099, V=100003, top=8, bits=16, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "logprobs"])
    if op == "norm":
        D = 8 * _log(rng, 16, 2048)
        norm = rng.random() < 0.75
        return dict(op=op, T=_log(rng, 1, min(16384, 16384 * 6144 // D)), D=D, residual=rng.random() < 0.7, norm=norm,
                    outs=rng.choice(["q", "bf16", "both"]), pad=rng.choice([0, 0, 8 * rng.randrange(1, 200)]))
    if op == "linear":
        M = _log(rng, 1, 16384)
        K = 16 * _log(rng, 4, 1024)
        N = _log(rng, 64, min(40000, 16384 * 18432 * 6144 // (4 * M * K)))
        act = rng.choice([None, None, "silu", "gelu", "silu_gated"])
        return dict(op=op, M=M, N=N + N % 2 if act == "silu_gated" else N, K=K, bits=rng.choice([8, 8, 16]), act=act,
                    bias=rng.random() < 0.4, residual=rng.random() < 0.4, out=rng.choice(["bf16", "bf16", "f32"]))
    T = rng.randrange(1, 9)
    V = _log(rng, 300, 200000)
    return dict(op=op, B=_log(rng, 1, max(1, min(1000, 200_000_000 // (V * T)))), T=T, V=V, top=rng.randrange(0, 33),
                bits=rng.choice([32, 32, 16]), ragged=rng.random() < 0.5)


# -------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _asked(case):
    """Rows of each sequence that a token is given for.  A case has the same counts for every seed (the order of the
    sequences is the seed's)."""
    rng = random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))
    return [rng.randint(1, case["T"]) if case["ragged"] else case["T"] for _ in range(case["B"])]


def _codes(rows, cols, g):
    """e4m3 codes with one scale per row, as a quantised matrix of about unit values has them."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    scale = x.abs().amax(-1) / E4M3_MAX
    return (x / scale[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case, op=case["op"])
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        # a residual stream has channels that are far larger than the rest
        wide = torch.exp(torch.randn(D, generator=g, device=DEV))
        s["x"] = torch.randn(T, D + case["pad"], generator=g, device=DEV).bfloat16()[:, :D]
        s["residual"] = (torch.randn(T, D, generator=g, device=DEV) * wide).bfloat16() if case["residual"] else None
        s["weight"] = 1 + 0.1 * torch.randn(D, generator=g, device=DEV) if case["norm"] else None
        like = dict(dtype=torch.bfloat16, device=DEV)
        s["residual_out"] = torch.zeros(T, D, **like) if case["residual"] else None
        s["out"] = torch.zeros(T, D, **like) if case["outs"] != "q" else None
        s["out_q"] = s["out_scale"] = None
        if case["outs"] != "bf16":
            s["out_q"] = torch.zeros(T, D, **like).to(torch.float8_e4m3fn)
            s["out_scale"] = torch.zeros(T, device=DEV)
        if own:
            from linear_attention_decode_04_gb300 import KdaAddNormCall
            s["call"] = KdaAddNormCall(s["x"], weight=s["weight"], residual=s["residual"],
                                       residual_out=s["residual_out"], out=s["out"], out_q=s["out_q"],
                                       out_scale=s["out_scale"], eps=EPS, norm=case["norm"])
        return s
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        width = N // 2 if case["act"] == "silu_gated" else N
        s["x_scale"] = s["weight_scale"] = None
        if case["bits"] == 8:
            s["x"], s["x_scale"] = _codes(M, K, g)
            s["weight"], s["weight_scale"] = _codes(N, K, g)
            s["weight_scale"] = s["weight_scale"] / math.sqrt(K)
        else:
            s["x"] = torch.randn(M, K, generator=g, device=DEV).bfloat16()
            s["weight"] = (torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K)).bfloat16()
        s["bias"] = torch.randn(N, generator=g, device=DEV) if case["bias"] else None
        s["residual"] = torch.randn(M, width, generator=g, device=DEV).bfloat16() if case["residual"] else None
        s["out"] = torch.zeros(M, width, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=DEV)
        if own:
            from linear_attention_decode_04_gb300 import KdaLinearCall
            s["call"] = KdaLinearCall(s["x"], s["weight"], s["out"], x_scale=s["x_scale"],
                                      weight_scale=s["weight_scale"], bias=s["bias"], residual=s["residual"],
                                      activation=case["act"], early_weight=True)
        return s
    B, T, V = case["B"], case["T"], case["V"]
    dt = torch.float32 if case["bits"] == 32 else torch.bfloat16
    s["logits"] = torch.empty(B * T, V, dtype=dt, device=DEV)
    tokens = torch.empty(B * T, dtype=torch.int32, device=DEV)
    for r in range(0, B * T, 512):     # (by parts: the random numbers take more room than the rows)
        z = torch.randn(min(512, B * T - r), V, generator=g, device=DEV) * 3
        z[::8, V // 3:V // 3 + V // 10] = float("-inf")          # rows of a constrained output: tokens ruled out
        z = z.to(dt)
        s["logits"][r:r + 512] = z
        # a token drawn from the row's probabilities
        u = torch.rand(z.shape, generator=g, device=DEV).clamp_(1e-20, 1 - 1e-7)
        tokens[r:r + 512] = (z.float() - u.log_().neg_().log_()).argmax(-1)
    s["logits"], s["tokens"] = s["logits"].view(B, T, V), tokens.view(B, T)
    n = _asked(case)
    random.Random(seed).shuffle(n)
    s["tokens"][torch.arange(T, device=DEV) >= torch.tensor(n, device=DEV)[:, None]] = -1
    if own:
        from linear_attention_decode_04_gb300 import KdaLogprobsCall
        s["call"] = KdaLogprobsCall(s["logits"], s["tokens"], num_top=case["top"])
    return s


# ---------------------------------------------------------------------- run
def run(s):
    if own:
        return _run_own(s)
    return dict(norm=_norm, linear=_linear, logprobs=_logprobs)[s["op"]](s)


def _norm_outputs(s):
    return {k: s[k] for k in ("residual_out", "out", "out_q", "out_scale") if s[k] is not None}


def _run_own(s):
    c = s["call"]
    c()
    if s["op"] == "norm":
        return _norm_outputs(s)
    if s["op"] == "linear":
        return dict(out=s["out"])
    return dict(logprobs=c.logprobs, ranks=c.ranks, entropy=c.entropy, top_ids=c.top_ids,
                top_logprobs=c.top_logprobs)


def _norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
        s["residual_out"].copy_(h)
    if s["case"]["norm"]:
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    if s["out"] is not None:
        s["out"].copy_(h)
    if s["out_q"] is not None:
        s["out_scale"].copy_(h.abs().amax(-1).clamp(min=SCALE_FLOOR) / E4M3_MAX)
        s["out_q"].copy_((h / s["out_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn))
    return _norm_outputs(s)


def _linear(s):
    act = s["case"]["act"]
    y = s["x"].float() @ s["weight"].float().t()
    if s["x_scale"] is not None:
        y = y * s["x_scale"][:, None] * s["weight_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if act == "silu":
        y = y / (1 + torch.exp(-y))
    elif act == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif act == "silu_gated":
        a, b = y.chunk(2, -1)
        y = a / (1 + torch.exp(-a)) * b
    if s["residual"] is not None:
        y = y + s["residual"].float()
    s["out"].copy_(y)
    return dict(out=s["out"])


def _logprobs(s):
    B, T, V = s["logits"].shape
    k = min(s["case"]["top"], V)
    x = s["logits"].view(B * T, V).float()
    tok = s["tokens"].view(-1).long()
    asked = tok >= 0
    at = tok.clamp(min=0)[:, None]
    top = x.amax(-1, keepdim=True)
    d = x - top
    e = torch.exp(d)
    total = e.sum(-1)
    lse = top[:, 0] + torch.log(total)
    entropy = torch.log(total) - (torch.where(e > 0, d, 0.0) * e).sum(-1) / total
    xt = x.gather(1, at)
    ids = torch.arange(V, device=DEV)
    ranks = ((x > xt) | ((x == xt) & (ids < at))).sum(-1)
    # whole numbers in the logits' order; among equal logits the lower index is larger
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long()
    best = torch.topk(order * 2 ** 32 + (2 ** 31 - 1 - ids), k, -1).values
    best = 2 ** 31 - 1 - (best & (2 ** 32 - 1))
    best_lp = x.gather(1, best) - lse[:, None]

    def shaped(v, absent, dt, width=()):
        v = torch.where(asked.view(-1, *([1] * len(width))), v, absent).to(dt)
        return v.view(B, T, *width)

    return dict(logprobs=shaped(xt[:, 0] - lse, 0.0, torch.float32), ranks=shaped(ranks, -1, torch.int32),
                entropy=shaped(entropy, 0.0, torch.float32), top_ids=shaped(best, -1, torch.int32, (k,)),
                top_logprobs=shaped(best_lp, 0.0, torch.float32, (k,)))


# --------------------------------------------------------------------- work
def work(case):
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        each = 2.0 + (4.0 if case["residual"] else 0.0) + dict(q=1.0, bf16=2.0, both=3.0)[case["outs"]]
        return {"bytes": T * D * each + 4.0 * D * case["norm"] + 4.0 * T * (case["outs"] != "bf16"),
                "flops": 6.0 * T * D}
    if case["op"] == "linear":
        M, N, K, b = case["M"], case["N"], case["K"], case["bits"] // 8
        width = N // 2 if case["act"] == "silu_gated" else N
        size = (2.0 if case["out"] == "bf16" else 4.0) + (2.0 if case["residual"] else 0.0)
        return {"bytes": 1.0 * b * K * (M + N) + M * width * size + 4.0 * N * case["bias"] + 4.0 * (M + N) * (b == 1),
                "flops": 2.0 * M * N * K}
    n = sum(_asked(case))
    return {"bytes": 1.0 * n * case["V"] * (case["bits"] // 8) + case["B"] * case["T"] * (16.0 + 8.0 * case["top"]),
            "flops": 5.0 * n * case["V"]}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return dict(norm=_exact_norm, linear=_exact_linear, logprobs=_exact_logprobs)[case["op"]](case, s)


def _exact_norm(case, s):
    h = s["x"].double()
    res = {}
    if case["residual"]:
        h = res["residual_out"] = h + s["residual"].double()
    if case["norm"]:
        h = torch.einsum("td,t,d->td", h, (h.pow(2).sum(-1) / case["D"] + EPS).pow(-0.5), s["weight"].double())
    if case["outs"] != "q":
        res["out"] = h
    if case["outs"] != "bf16":
        top = torch.maximum(h.amax(-1), -h.amin(-1))
        res["out_scale"] = torch.where(top > SCALE_FLOOR, top, SCALE_FLOOR) / E4M3_MAX
        res["out_q"] = h / res["out_scale"][:, None]         # what the codes stand for, before it is rounded to them
    return {k: res[k] for k in ("residual_out", "out", "out_q", "out_scale") if k in res}


def _exact_linear(case, s):
    w = s["weight"].double()
    if case["bits"] == 8:
        w = w * s["weight_scale"].double()[:, None]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
    for m in range(0, case["M"], 2048):
        x = s["x"][m:m + 2048].double()
        if case["bits"] == 8:
            x = x * s["x_scale"][m:m + 2048].double()[:, None]
        y = torch.einsum("mk,nk->mn", x, w)
        if case["bias"]:
            y += s["bias"].double()
        if case["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif case["act"] == "gelu":
            y = y * (1 - 0.5 * torch.special.erfc(y / math.sqrt(2)))
        elif case["act"] == "silu_gated":
            h = case["N"] // 2
            y = y[:, :h] * torch.sigmoid(y[:, :h]) * y[:, h:]
        out[m:m + 2048] = y
        if case["residual"]:
            out[m:m + 2048] += s["residual"][m:m + 2048].double()
    return dict(out=out)


def _exact_logprobs(case, s):
    B, T, V = s["logits"].shape
    k = min(case["top"], V)
    rows, tok = s["logits"].view(B * T, V), s["tokens"].view(-1)
    lp = torch.zeros(B * T, dtype=torch.float64, device=DEV)
    entropy, ranks = lp.clone(), torch.full_like(lp, -1).int()
    ids, best = torch.full((B * T, k), -1, dtype=torch.int32, device=DEV), lp.new_zeros(B * T, k)
    live = torch.nonzero(tok >= 0)[:, 0]
    for part in live.split(128):
        x = rows[part].double()
        t = tok[part].long()
        lse = torch.logsumexp(x, -1, keepdim=True)
        entropy[part] = torch.special.entr(torch.exp(x - lse)).sum(-1)
        lp[part] = (x.gather(1, t[:, None]) - lse)[:, 0]
        z, order = torch.sort(x, stable=True, dim=-1, descending=True)
        ranks[part] = (order == t[:, None]).int().argmax(-1).int()
        ids[part], best[part] = order[:, :k].int(), z[:, :k] - lse
    return dict(logprobs=lp.view(B, T), ranks=ranks.view(B, T), entropy=entropy.view(B, T), top_ids=ids.view(B, T, k),
                top_logprobs=best.view(B, T, k))
