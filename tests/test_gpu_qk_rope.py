"""Per-head norm, rotation and 8-bit cache write against the 64-bit reference.

Tolerances, from the roundings alone.  The kernel works in fp32: the sum of
128 squares, the reciprocal root and the products stay within 2^-20 relative
of the exact normed value; the rotation's sine and cosine are off by at most
2^-22 and multiply values of at most the row's largest.  So a value x of a
row whose largest is m is within FP32 * m, FP32 = 2^-19, before its last
rounding: half a step of bf16 (2^-8 |x|), or of e4m3 (2^-4 |x|, or 2^-10
scales in the subnormal range)."""
import numpy as np
import pytest
import torch

import step_reference as R
from linear_attention_decode_04_gb300 import KdaQkRopeCall, kda_qk_rope, rope_frequencies

pytestmark = pytest.mark.gpu
FP32 = 2.0 ** -19


def slots_of(rng, ctx, new, bs, spare=2):
    """slot map of requests with ctx cached and new tokens; blocks drawn without order"""
    pages = [-(-(c % bs + n) // bs) for c, n in zip(ctx, new)]
    perm = rng.permutation(sum(pages) + spare)
    slot, at = [], 0
    for c, n, k in zip(ctx, new, pages):
        slot += [int(perm[at + (c % bs + j) // bs]) * bs + (c + j) % bs for j in range(n)]
        at += k
    return slot, len(perm)


class Case:
    def __init__(self, dev, Hq, Hkv, ctx, new, bs=16, rot=128, inter=False, seed=0, pad=0, weights=True, cache=True,
                 k_out=False, row_pad=0, scale=1.0, base=1e6):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.__dict__.update(dev=dev, Hq=Hq, Hkv=Hkv, bs=bs, rot=rot, inter=inter, base=base)
        self.pos = [c + j for c, n in zip(ctx, new) for j in range(n)] + [0] * pad
        self.T = T = len(self.pos)
        self.slot, self.nb = slots_of(rng, ctx, new, bs)
        self.slot += [-1] * pad
        W = (Hq + 2 * Hkv) * 128
        self.qkv = torch.zeros(T, W + row_pad, dtype=torch.bfloat16, device=dev)[:, :W]
        self.qkv.copy_((torch.randn(T, W, generator=g) * scale).bfloat16())
        self.wq = 1 + 0.1 * torch.randn(128, generator=g) if weights else None
        self.wk = 1 + 0.1 * torch.randn(128, generator=g) if weights else None
        self.q_out = torch.full((T, Hq * 128 + row_pad), 5.0, dtype=torch.bfloat16, device=dev)[:, :Hq * 128]
        self.k_out = torch.full((T, Hkv * 128), 5.0, dtype=torch.bfloat16, device=dev) if k_out else None
        self.cache = cache
        if cache:
            shape = (self.nb, Hkv, bs, 128)
            self.codes = [torch.randint(0, 256, shape, generator=g, dtype=torch.int32) for _ in "kv"]
            self.codes = [torch.where(c & 127 == 127, c - 1, c).to(torch.uint8) for c in self.codes]   # no NaN codes
            self.scales = [torch.exp2(torch.randint(-9, -2, (self.nb, Hkv), generator=g).float()) for _ in "kv"]
            self.gcodes = [c.to(dev).view(torch.float8_e4m3fn) for c in self.codes]
            self.gscales = [s.to(dev) for s in self.scales]

    def kwargs(self):
        t = lambda v, dt: torch.tensor(v, dtype=dt, device=self.dev)  # noqa: E731
        kw = dict(num_q_heads=self.Hq, num_kv_heads=self.Hkv, rope_freqs=rope_frequencies(self.rot, self.base, self.dev),
                  interleaved=self.inter, k_out=self.k_out,
                  q_weight=None if self.wq is None else self.wq.to(self.dev),
                  k_weight=None if self.wk is None else self.wk.to(self.dev),
                  err_flag=torch.zeros(1, dtype=torch.int32, device=self.dev))
        if self.cache:
            kw.update(k_cache=self.gcodes[0], v_cache=self.gcodes[1], k_scale=self.gscales[0], v_scale=self.gscales[1],
                      slot_map=t(self.slot, torch.int64))
        return (self.qkv, t(self.pos, torch.int32), self.q_out), kw

    def check(self, err=0, x=None):
        args, kw = self.kwargs()
        x = self.qkv.cpu().double().numpy().reshape(self.T, self.Hq + 2 * self.Hkv, 128) if x is None else x
        kda_qk_rope(*args, **kw)
        torch.cuda.synchronize(self.dev)
        assert kw["err_flag"].item() == err
        self.compare(x)

    def compare(self, x):
        f = R.inv_freqs(self.rot, self.base)
        w = [None if v is None else v.numpy() for v in (self.wq, self.wk)]
        Hq, Hkv = self.Hq, self.Hkv
        q = np.stack([R.norm_rotate(x[t, :Hq], w[0], self.pos[t], f, self.inter, 1e-6) for t in range(self.T)]) \
            if self.T else np.zeros((0, Hq, 128))
        k = np.stack([R.norm_rotate(x[t, Hq:Hq + Hkv], w[1], self.pos[t], f, self.inter, 1e-6) for t in range(self.T)]) \
            if self.T else np.zeros((0, Hkv, 128))
        for got, want in ((self.q_out, q), (self.k_out, k)):
            if got is not None:
                got = got.cpu().double().numpy().reshape(want.shape)
                lim = 2.0 ** -8 * np.abs(want) + FP32 * np.abs(want).max(-1, keepdims=True) + 1e-30
                assert (np.abs(got - want) <= lim).all(), np.abs(got - want).max()
        if not self.cache:
            return
        live = [s if 0 <= s < self.nb * self.bs else -1 for s in self.slot]
        for i, y in enumerate((k, x[:, Hq + Hkv:])):
            codes, scale, new = R.write_cache(self.codes[i].numpy(), self.scales[i].numpy(), y, live, self.bs)
            got, gs = self.gcodes[i].view(torch.uint8).cpu().numpy(), self.gscales[i].cpu().double().numpy()
            assert np.array_equal(gs, scale)
            vals = R.e4m3_values()
            for (b, h), rows in new.items():
                for r, want in rows:
                    have, s = vals[got[b, h, r]] * scale[b, h], scale[b, h]
                    m = np.abs(want).max()
                    lim = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s) + FP32 * m
                    assert (np.abs(have - want) <= lim).all(), (b, h, r)
                    codes[b, h, r] = got[b, h, r]
            assert np.array_equal(got, codes)      # older rows rescaled exactly, all else untouched


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("inter", [False, True])
def test_blocks_and_runs(bs, inter, cuda_device):
    # new blocks, runs that start and end inside a block, runs over several blocks, a run of one
    ctx = [0, 5, bs - 1, bs, 3 * bs + 7, 0, bs // 2]
    new = [1, 3, 2, 1, 2 * bs + 5, bs, bs // 2]
    Case(cuda_device, 6, 2, ctx, new, bs=bs, rot=64, inter=inter, seed=bs, pad=3, k_out=True).check()


@pytest.mark.parametrize("rot", [0, 16, 48, 112, 128])
@pytest.mark.parametrize("inter", [False, True])
def test_rotary_widths(rot, inter, cuda_device):
    Case(cuda_device, 5, 1, [7, 100], [3, 2], rot=rot, inter=inter, seed=rot, k_out=True).check()


@pytest.mark.parametrize("Hq, Hkv", [(1, 1), (7, 7), (33, 11), (96, 8), (16, 1)])
def test_head_layouts(Hq, Hkv, cuda_device):
    Case(cuda_device, Hq, Hkv, [0, 9], [4, 1], seed=Hq, row_pad=8).check()


def test_far_positions(cuda_device):
    # angles of positions up to 2^31: the reference's own angle is good to 2^31 * 2^-53 turns
    for pos in (10 ** 6, 2 ** 30, 2 ** 31 - 5):
        Case(cuda_device, 4, 2, [pos], [3], bs=16, rot=128, seed=3).check()


def test_without_norm_cache_or_rotation(cuda_device):
    Case(cuda_device, 4, 2, [3], [5], weights=False, seed=1).check()
    Case(cuda_device, 4, 2, [3], [5], cache=False, k_out=True, seed=2).check()
    Case(cuda_device, 4, 2, [3], [5], weights=False, rot=0, cache=False, k_out=True, seed=3).check()
    Case(cuda_device, 4, 0, [3], [5], cache=False, seed=4).check()
    Case(cuda_device, 4, 2, [], [], cache=False, seed=5).check()            # no rows
    c = Case(cuda_device, 4, 2, [3], [5], seed=6)
    c.wk = None                                                             # queries normed, keys not
    c.check()


def test_prompt_sized_batches(cuda_device):
    # enough rows that a CTA looks through several and a warp takes all heads of a token
    Case(cuda_device, 4, 2, [0, 77, 31], [5000, 900, 1], bs=64, rot=64, seed=9).check()
    Case(cuda_device, 3, 1, [5], [9000], bs=16, rot=128, inter=True, seed=10).check()


def test_in_place_queries_and_keys(cuda_device):
    c = Case(cuda_device, 4, 2, [0, 40], [7, 2], seed=21)
    x = c.qkv.cpu().double().numpy().reshape(c.T, -1, 128)
    c.q_out = c.qkv[:, :4 * 128]
    c.check(x=x)
    c = Case(cuda_device, 4, 2, [0, 40], [7, 2], seed=22, cache=False)
    x = c.qkv.cpu().double().numpy().reshape(c.T, -1, 128)
    c.q_out, c.k_out = c.qkv[:, :4 * 128], c.qkv[:, 4 * 128:6 * 128]
    c.check(x=x)


def test_scale_grows_and_never_shrinks(cuda_device):
    # a block filled a token at a time, with values that grow, then shrink: the same block again and again
    dev, bs = cuda_device, 16
    for growth in (4.0, 0.25):
        c = Case(dev, 2, 2, [0], [1], bs=bs, weights=False, seed=31)
        for r in range(bs):
            c.slot, c.pos = [c.slot[0] // bs * bs + r], [r]
            c.qkv.copy_((torch.randn(c.qkv.shape, generator=torch.Generator().manual_seed(r)) * growth ** (r / 3)).bfloat16())
            c.codes = [v.view(torch.uint8).cpu().clone() for v in c.gcodes]
            c.scales = [v.cpu().clone() for v in c.gscales]
            c.check()


def test_values_at_the_edges_of_the_format(cuda_device):
    c = Case(cuda_device, 2, 2, [0, 3], [4, 2], bs=16, rot=0, weights=False, seed=41)
    x = c.qkv.view(c.T, 6, 128)
    x[0] = 0.0                                                # zeros only in the first rows
    x[1, 4:, 5] = 3.0e38                                      # beyond the largest scale: saturates
    x[2, 2:, 7] = 1e-38
    x[4] = 0.0                                                # a run that is all zero behind older rows
    x[5] = 0.0
    args, kw = c.kwargs()
    x64 = c.qkv.cpu().double().numpy().reshape(c.T, -1, 128)
    x64 = np.where(np.abs(x64) > 448 * 2.0 ** 119, 448 * 2.0 ** 119 * np.sign(x64), x64)
    kda_qk_rope(*args, **kw)
    torch.cuda.synchronize()
    c.q_out, keep = None, c.q_out
    c.compare(x64)
    c.q_out = keep
    # not finite: NaN stays NaN, infinities saturate, neither counts for the scale
    c = Case(cuda_device, 2, 2, [0], [3], bs=16, rot=0, weights=False, seed=42)
    x = c.qkv.view(c.T, 6, 128)
    x[0, 2:, 3], x[1, 2:, 4], x[2, 2:, 9] = float("nan"), float("inf"), float("-inf")
    args, kw = c.kwargs()
    kda_qk_rope(*args, **kw)
    b = c.slot[0] // 16
    for codes, scale, part in ((c.gcodes[0], c.gscales[0], x[:, 2:4]), (c.gcodes[1], c.gscales[1], x[:, 4:])):
        v = codes[b].float()
        assert v[:, 0, 3].isnan().all() and (v[:, 1, 4] == 448).all() and (v[:, 2, 9] == -448).all()
        assert v.isnan().sum() == 2
        fin = torch.where(part.isfinite(), part.float(), torch.zeros(())).abs().amax((0, 2)).tolist()
        assert scale[b].tolist() == [R.fit_scale(f) for f in fin]


def test_cache_layouts_by_stride(cuda_device):
    # [blocks, rows, heads, 128] and blocks that hold K and V together, through strided views
    dev, Hkv, bs = cuda_device, 3, 16
    for kind in ("token_major", "joined"):
        c = Case(dev, 3, Hkv, [4, 0], [20, 3], bs=bs, seed=51)
        if kind == "token_major":
            base = [torch.zeros(c.nb, bs, Hkv, 128, dtype=torch.uint8, device=dev) for _ in "kv"]
            view = [b.transpose(1, 2).view(torch.float8_e4m3fn) for b in base]
        else:
            base = torch.zeros(c.nb, 2, Hkv, bs, 128, dtype=torch.uint8, device=dev)
            view = [base[:, i].view(torch.float8_e4m3fn) for i in range(2)]
        for v, code in zip(view, c.codes):
            v.view(torch.uint8).copy_(code.to(dev))
        c.gcodes = view
        c.check()


def test_slots_out_of_range(cuda_device):
    c = Case(cuda_device, 2, 1, [0, 16], [5, 2], seed=61)
    args, kw = c.kwargs()
    before = [v.view(torch.uint8).clone() for v in c.gcodes]
    kda_qk_rope(*args, **{**kw, "slot_map": torch.tensor([c.nb * 16, 2 ** 40, 2 ** 62, -1, -7, -2 ** 40, -1], device=cuda_device)})
    torch.cuda.synchronize()
    assert kw["err_flag"].item() == R.SLOT_RANGE
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, c.gcodes))


def test_graph_replay_and_stream(cuda_device):
    c = Case(cuda_device, 4, 2, [3, 30], [2, 2], seed=71)
    args, kw = c.kwargs()
    call = KdaQkRopeCall(*args, **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    g.replay()
    torch.cuda.synchronize()
    c.compare(c.qkv.cpu().double().numpy().reshape(c.T, -1, 128))
    s = torch.cuda.Stream()
    c = Case(cuda_device, 4, 2, [3, 30], [2, 2], seed=72)
    args, kw = c.kwargs()
    s.wait_stream(torch.cuda.current_stream())
    kda_qk_rope(*args, **kw, stream=s)
    s.synchronize()
    c.compare(c.qkv.cpu().double().numpy().reshape(c.T, -1, 128))


def test_refusals(cuda_device):
    c = Case(cuda_device, 4, 2, [3], [2], seed=81)
    args, kw = c.kwargs()
    bad = [dict(slot_map=None), dict(num_q_heads=5), dict(k_scale=kw["k_scale"][:, :1]), dict(q_weight=kw["q_weight"].double()),
           dict(k_cache=kw["k_cache"].view(torch.uint8)), dict(k_cache=kw["k_cache"][:, :, :8]),
           dict(v_cache=kw["v_cache"][:1]), dict(slot_map=kw["slot_map"].int()), dict(slot_map=kw["slot_map"][:1])]
    for b in bad:
        with pytest.raises((ValueError, TypeError)):
            kda_qk_rope(*args, **{**kw, **b})
    with pytest.raises(Exception, match="k_out"):
        kda_qk_rope(*args, **{**kw, "k_out": c.qkv[:, 512:768]})
    with pytest.raises(Exception, match="rot_dim"):
        kda_qk_rope(*args, **{**kw, "rope_freqs": torch.zeros(4, dtype=torch.int64, device=cuda_device)})


@pytest.mark.parametrize("Hq, Hkv, bs, inter", [(22, 3, 16, False), (40, 1, 256, True), (33, 2, 64, False)])
def test_large_batches_give_the_bits_of_small_ones(Hq, Hkv, bs, inter, cuda_device):
    # every SM several times over, other splits of rows and heads over CTAs; the last group of heads not whole
    T = 2 * 152 * 24 + 5
    g = torch.Generator(device=cuda_device).manual_seed(Hq)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * 128 + 64, device=cuda_device, generator=g).bfloat16()
    w = torch.rand(2, 128, device=cuda_device, generator=g) + 0.5
    pos = torch.randint(0, 10 ** 6, (T,), device=cuda_device, generator=g, dtype=torch.int32)
    nb = -(-T // bs)
    kw = dict(num_q_heads=Hq, num_kv_heads=Hkv, rope_freqs=rope_frequencies(96, 1e4, cuda_device), interleaved=inter,
              q_weight=w[0], k_weight=w[1])

    def run(rows):
        n = rows.numel()
        q, k = (torch.full((n, h * 128), 9.0, dtype=torch.bfloat16, device=cuda_device) for h in (Hq, Hkv))
        cache = [torch.zeros(nb, Hkv, bs, 128, dtype=torch.uint8, device=cuda_device).view(torch.float8_e4m3fn) for _ in "kv"]
        scale = [torch.zeros(nb, Hkv, device=cuda_device) for _ in "kv"]
        err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        kda_qk_rope(qkv[rows], pos[rows], q, k_out=k, k_cache=cache[0], v_cache=cache[1], k_scale=scale[0], v_scale=scale[1],
                    slot_map=rows, err_flag=err, **kw)
        assert err.item() == 0
        return q, k, [c.view(torch.uint8) for c in cache], scale
    rows = torch.arange(T, device=cuda_device)
    q, k, cache, scale = run(rows)
    # the same rows in small batches (tested above against 64 bits)
    step = 2048
    for t in range(0, T, step):
        part = rows[t:t + step]
        q2, k2, cache2, scale2 = run(part)
        assert torch.equal(q[t:t + step], q2) and torch.equal(k[t:t + step], k2)
        b0, b1 = t // bs, -(-min(t + step, T) // bs)
        for a, b in zip(cache + scale, cache2 + scale2):
            assert torch.equal(a[b0:b1], b[b0:b1])
    # in place
    x = qkv.clone()
    kda_qk_rope(x, pos, x[:, :Hq * 128], **kw)
    assert torch.equal(x[:, :Hq * 128], q) and torch.equal(x[:, Hq * 128:], qkv[:, Hq * 128:])
