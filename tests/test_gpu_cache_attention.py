"""Attention over the 8-bit paged cache against a 64-bit softmax attention.

Tolerance, from the roundings alone.  Write a_s for the exact softmax weights
and |v|_a = sum_s a_s |v_s|.
- q enters as two e4m3 parts: exact down to 2^-10 steps of a row scaled to
  (224, 448], i.e. off by at most 2^-18 of the row's largest |q|; with fp32
  accumulation of 128 products a logit is off by at most
  E = (2^-18 + 2^-17) * sm_scale * max|q| * sum_d |k_d| (+ 2^-22 |logit|).
- a weight is rounded to fp16 (2^-12) and then to two e4m3 parts: relative
  error 2^-8 (half a step of the second part, itself at most half a step of
  the first), or absolutely at most 2^-18 of the largest weight of its tile.
- out is rounded to bf16 (2^-8 |out|).
So |got - out| <= 2^-8 |out| + (2^-8 + 2^-11 + 2 E) |v|_a + 2^-18 * 128 *
tile-wise largest |v| contribution; the last is bounded with
2^-11 * max_s a_s |v|_max per tile, below 2^-10 sum of tiles' largest
weights times the largest |v|.  Masks are exact: what no query sees must
not matter at all."""
import math

import numpy as np
import pytest
import torch

import step_reference as R
from linear_attention_decode_04_gb300 import KdaCacheAttentionCall, cache_attention_workspace, kda_cache_attention

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, dev, lens, new, Hq=8, Hkv=2, bs=16, seed=0, scale_q=1.0, scales=(-7, -4), extra=0, row_pad=0,
                 garbage=True, layout="head", table_pad=2, outlier=False):
        g = torch.Generator().manual_seed(seed)
        self.dev, self.lens, self.new, self.Hq, self.Hkv, self.bs = dev, list(lens), list(new), Hq, Hkv, bs
        B, G = len(lens), Hq // Hkv
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)
        self.T = T = self.cu[-1] + extra
        pages = [-(-max(n, 0) // bs) for n in lens]
        nb = sum(pages) + 3
        perm = torch.randperm(nb, generator=g).tolist()
        M = max(pages + [1]) + table_pad
        self.table = torch.full((B, M), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.table[b, :pages[b]] = torch.tensor(perm[at:at + pages[b]], dtype=torch.int32)
            at += pages[b]
        shape = (nb, Hkv, bs, 128)
        rnd = lambda: (torch.randn(shape, generator=g) * 60).clamp(-440, 440).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        self.k, self.v = rnd(), rnd()
        if outlier:                       # some tokens far above the rest, some values too
            self.k[:, :, 3] = torch.tensor(440.0).to(torch.float8_e4m3fn).view(torch.uint8)
        self.ks = torch.exp2(torch.randint(*scales, (nb, Hkv), generator=g).float())
        self.vs = torch.exp2(torch.randint(*scales, (nb, Hkv), generator=g).float())
        if garbage:                       # NaN codes in every row behind a sequence's end, and in unused blocks
            used = torch.zeros(nb, bs, dtype=torch.bool)
            for b in range(B):
                for p in range(pages[b]):
                    used[self.table[b, p], :min(bs, lens[b] - p * bs)] = True
            for c in (self.k, self.v):
                c[~used.unsqueeze(1).expand(nb, Hkv, bs)] = 0x7f
        self.q = (torch.randn(T, Hq * 128, generator=g) * scale_q).bfloat16()
        self.row_pad, self.layout, self.nb = row_pad, layout, nb
        self.sm = 0.0

    def tensors(self):
        d = self.dev
        wide = lambda t: torch.cat([t, t.new_zeros(t.shape[0], self.row_pad)], 1).to(d)[:, :t.shape[1]]  # noqa: E731

        def cache(c):
            if self.layout == "token":    # [blocks, rows, heads, 128] in memory
                return c.transpose(1, 2).contiguous().to(d).transpose(1, 2).view(torch.float8_e4m3fn)
            return c.to(d).view(torch.float8_e4m3fn)
        i = lambda v: torch.tensor(v, dtype=torch.int32, device=d)  # noqa: E731
        out = torch.full((self.T, self.Hq * 128 + self.row_pad), 7.0, dtype=torch.bfloat16, device=d)[:, :self.Hq * 128]
        return (wide(self.q), i(self.cu), i(self.lens), self.table.to(d), cache(self.k), cache(self.v), self.ks.to(d),
                self.vs.to(d), out)

    def reference(self):
        """(out, allowed error) fp64 [T, Hq, 128]; rows outside every sequence NaN"""
        Hq, Hkv, bs, G = self.Hq, self.Hkv, self.bs, self.Hq // self.Hkv
        vals = torch.from_numpy(R.e4m3_values())
        sm = self.sm or 1 / math.sqrt(128)
        out = torch.full((self.T, Hq, 128), float("nan"), dtype=torch.float64)
        tol = torch.zeros_like(out)
        for b, (n, m) in enumerate(zip(self.lens, self.new)):
            n = max(n, 0)
            ids = self.table[b, :-(-n // bs)].long()
            k, v = ((vals[c[ids].long()] * s[ids].double()[..., None, None]).transpose(0, 1).reshape(Hkv, -1, 128)[:, :n]
                    for c, s in ((self.k, self.ks), (self.v, self.vs)))
            q = self.q[self.cu[b]:self.cu[b + 1]].double().view(m, Hkv, G, 128)
            for j in range(m):
                lim = max(0, min(n, self.lens[b] - m + j + 1))
                t = self.cu[b] + j
                if lim == 0:
                    out[t] = 0
                    continue
                z = torch.einsum("hgd,hld->hgl", q[j], k[:, :lim]) * sm
                a = torch.softmax(z, -1)
                o = torch.einsum("hgl,hld->hgd", a, v[:, :lim])
                av = torch.einsum("hgl,hld->hgd", a, v[:, :lim].abs())
                # the error of a logit is sm times that of q . k, so its bound has |sm| (a bound is not negative)
                e = (2.0 ** -18 + 2.0 ** -17) * abs(sm) * q[j].abs().amax(-1, keepdim=True) * k[:, :lim].abs().sum(-1).amax(-1)[:, None, None]
                e = e + 2.0 ** -21 * z.abs().amax(-1, keepdim=True)
                pad = (-lim) % 128
                tile = torch.nn.functional.pad(a * v[:, :lim].abs().amax(-1)[:, None], (0, pad)).view(Hkv, G, -1, 128)
                small = 2.0 ** -10 * tile.amax(-1).sum(-1, keepdim=True)
                out[t] = o.reshape(Hq, 128)
                tol[t] = (2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -11 + 2 * e) * av + small).reshape(Hq, 128) + 1e-30
        return out, tol

    def check(self, max_new=None, err=0, ws=None):
        t = self.tensors()
        flag = torch.zeros(1, dtype=torch.int32, device=self.dev)
        ws = cache_attention_workspace(self.Hq, self.Hkv, max_new or max(self.new + [1]), self.dev) if ws is None else ws
        kda_cache_attention(*t, max_new=max_new or max(self.new + [1]), sm_scale=self.sm, err_flag=flag, workspace=ws)
        torch.cuda.synchronize(self.dev)
        assert flag.item() == err
        assert not ws[:1024].any()
        return self.compare(t[-1])

    def compare(self, out):
        want, tol = self.reference()
        got = out.cpu().double().view(self.T, self.Hq, 128)
        live = self.cu[-1]
        assert (got[live:] == 7.0).all()
        d = (got - want)[:live].abs()
        assert not d.isnan().any()
        assert (d <= tol[:live]).all(), f"{d.max():.3g}, {(d / tol[:live]).max():.3g} of the tolerance"
        return (d.norm() / want[:live].norm()).item() if live else 0.0


def test_one_tile(cuda_device):
    assert Case(cuda_device, [100], [1], Hq=1, Hkv=1, bs=128).check() < 4e-3
    assert Case(cuda_device, [100], [1], Hq=16, Hkv=1, bs=16).check() < 4e-3


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("Hq, Hkv, new", [(4, 4, 1), (12, 4, 1), (16, 2, 2), (24, 2, 2), (48, 8, 4), (33, 11, 3), (32, 1, 8)])
def test_steps(bs, Hq, Hkv, new, cuda_device):
    # every row tile (16, 32, 64 rows, and several tiles of 64); lengths around the 128 tokens of a tile
    # (that was with the first kernel's tiles: these are now 1, 3, 16, 24, 24, 9 and 256 rows, the variants of 8, 16 and 24
    # rows and the one for prompts; test_every_row_tile_at_every_block_size has all variants)
    lens = [new, 127, 128, 129, 1, 300, 1025]
    lens = [max(n, new) for n in lens]
    c = Case(cuda_device, lens, [new] * len(lens), Hq, Hkv, bs, seed=bs + Hq, row_pad=8, extra=2)
    assert c.check() < 4e-3


@pytest.mark.parametrize("Hq, Hkv", [(6, 2), (48, 8), (5, 5)])
def test_prompt_chunks(Hq, Hkv, cuda_device):
    # many row tiles per sequence; chunks with and without cached tokens before them; single tokens among them
    c = Case(cuda_device, [200, 333, 70, 1, 515], [200, 150, 1, 1, 97], Hq, Hkv, 32, seed=Hq)
    assert c.check() < 4e-3


def test_long_context_is_split_and_joined(cuda_device):
    # more tiles than CTAs for one sequence, beside short ones: every CTA takes part in several units
    c = Case(cuda_device, [50001, 3, 700, 20000], [1, 1, 1, 1], 4, 1, 64, seed=5)
    assert c.check() < 4e-3
    c = Case(cuda_device, [9000, 3, 4100], [6, 2, 8], 24, 3, 16, seed=6)
    assert c.check() < 4e-3


def test_rows_without_keys(cuda_device):
    # no tokens at all, fewer tokens than queries, a negative length, sequences without queries
    c = Case(cuda_device, [0, 2, 5, 64, 0, 130], [1, 4, 0, 3, 5, 2], 8, 2, 16, seed=7, extra=1)
    c.check()
    c.lens[4] = -3
    c.check()


def test_every_query_row_is_its_own_limit(cuda_device):
    # chunk longer than a tile of tokens from position 0: the first queries see 1, 2, 3 .. tokens
    assert Case(cuda_device, [300], [300], 2, 1, 16, seed=8).check() < 4e-3


def test_nan_values_reach_exactly_the_rows_that_see_them(cuda_device):
    for Hq, new in ((8, 4), (24, 8)):        # one and two groups of rows
        c = Case(cuda_device, [130, 260], [new, new], Hq, 2, 16, seed=9)
        # NaN in two channels of a value that only the last two queries see, and in one that all see
        c.v.view(torch.uint8)[c.table[0, 128 // 16].long(), 0, 0, 5] = 0x7f          # position 128 of 130
        c.v.view(torch.uint8)[c.table[0, 128 // 16].long(), 1, 0, 77] = 0xff
        c.v.view(torch.uint8)[c.table[1, 0].long(), 0, 3, 9] = 0x7f                  # position 3
        t = c.tensors()
        kda_cache_attention(*t, max_new=new)
        got = t[-1].cpu().double().view(c.T, 2, Hq // 2, 128)
        nan = torch.zeros_like(got, dtype=torch.bool)
        nan[new - 2:new, 0, :, 5] = True
        nan[new - 2:new, 1, :, 77] = True
        nan[new:, 0, :, 9] = True
        assert torch.equal(got.isnan(), nan)
        # the others are as if the values were finite
        c.v = torch.where(c.v & 0x7f == 0x7f, torch.zeros_like(c.v), c.v)
        want, tol = c.reference()
        ok = (got - want.view_as(got)).abs() <= tol.view_as(got)
        assert ok[~nan].all()


def test_nan_and_infinite_queries_and_keys(cuda_device):
    c = Case(cuda_device, [100, 40], [1, 2], 8, 2, 16, seed=10)
    c.q[0, 3] = float("nan")                                # head 0 of row 0
    c.q[1, 128 * 5 + 1] = float("inf")                      # head 5 of row 1
    c.k.view(torch.uint8)[c.table[1, 39 // 16].long(), 0, 39 % 16, 8] = 0x7f   # the last token: only row 2 sees it
    t = c.tensors()
    kda_cache_attention(*t, max_new=2)
    got = t[-1].float().cpu().view(3, 8, 128)
    bad = torch.zeros(3, 8, dtype=torch.bool)
    bad[0, 0] = bad[1, 5] = True
    bad[2, :4] = True
    assert torch.equal(got.isnan().all(-1), bad) and torch.equal(got.isnan().any(-1), bad)


@pytest.mark.parametrize("new", [3, 12])
def test_rows_that_are_not_finite_and_see_nothing_are_zero(new, cuda_device):
    c = Case(cuda_device, [1, 40], [new, 1], 8, 2, 16, seed=21)  # all but the first sequence's last query see nothing
    c.q[0, 5] = float("nan")
    c.q[1, 128 * 5 + 1] = float("inf")
    t = c.tensors()
    kda_cache_attention(*t, max_new=new)
    got = t[-1].float().cpu()
    assert (got[:new - 1] == 0).all() and not got.isnan().any() and (got[new - 1:new + 1] != 0).any(-1).all()


def test_scales_of_very_different_size(cuda_device):
    # V scales from 2^-40 to 2^20 in one sequence, K scales that make logits of +-100 and of 1e-6
    c = Case(cuda_device, [700, 300], [2, 1], 8, 2, 16, seed=11)
    g = torch.Generator().manual_seed(1)
    c.vs = torch.exp2(torch.randint(-40, 20, c.vs.shape, generator=g).float())
    c.check()
    c.ks = torch.exp2(torch.randint(-30, 1, c.ks.shape, generator=g).float())
    c.check()
    c.vs[:] = 2.0 ** -64                                    # what a block of zeros gets
    c.check()
    c.vs = 0.001 + torch.rand(c.vs.shape, generator=g)      # not powers of two
    c.check()


@pytest.mark.parametrize("scale_q, sm", [(1e-3, 0.0), (30.0, 0.0), (1.0, 1.0), (1e4, 1e-5), (1e-30, 1e29)])
def test_query_and_softmax_scales(scale_q, sm, cuda_device):
    c = Case(cuda_device, [300, 129], [1, 3], 12, 4, 32, seed=12, scale_q=scale_q)
    c.sm = sm
    c.check()


def test_one_token_far_above_the_rest(cuda_device):
    # most weights far below a tile's largest: the many small ones still count together
    c = Case(cuda_device, [4096], [1], 4, 1, 16, seed=13, outlier=True)
    c.check()
    c = Case(cuda_device, [20000], [1], 4, 1, 16, seed=14)
    c.k[:] = 0
    c.k[c.table[0, 0].long(), 0, 0] = 0x38                  # ones: the first token alone has a logit
    c.ks[:] = 1.0
    c.q[:] = 1.0
    c.sm = 9.0 / 128                                        # e^9 against 20,000 weights of 1
    c.check()


def test_head_layouts_and_strides(cuda_device):
    for layout in ("head", "token"):
        assert Case(cuda_device, [100, 260], [1, 3], 12, 4, 16, seed=15, layout=layout, row_pad=24).check() < 4e-3
    # K and V halves of one allocation
    c = Case(cuda_device, [100, 260], [1, 3], 12, 4, 32, seed=16)
    t = list(c.tensors())
    both = torch.stack([t[4].view(torch.uint8), t[5].view(torch.uint8)], 1)
    t[4], t[5] = both[:, 0].view(torch.float8_e4m3fn), both[:, 1].view(torch.float8_e4m3fn)
    kda_cache_attention(*t, max_new=3)
    assert c.compare(t[-1]) < 4e-3


def test_offsets_past_32_bits(cuda_device):
    # the blocks in use lie 5 GiB into the cache
    c = Case(cuda_device, [1000, 77], [1, 2], 8, 2, 64, seed=17, garbage=False)
    t = list(c.tensors())
    per = 2 * 64 * 128
    far = 5 * 2 ** 30 // per
    for i in (4, 5):
        big = torch.empty(far + c.nb, 2, 64, 128, dtype=torch.uint8, device=cuda_device)
        big[far:] = t[i].view(torch.uint8)
        t[i] = big.view(torch.float8_e4m3fn)
    for i in (6, 7):
        t[i] = torch.cat([torch.zeros(far, 2, device=cuda_device), t[i]])
    t[3] = torch.where(t[3] >= 0, t[3] + far, t[3])
    kda_cache_attention(*t, max_new=2)
    assert c.compare(t[-1]) < 4e-3


def test_bad_blocks_count_as_absent(cuda_device):
    c = Case(cuda_device, [200, 90], [1, 1], 4, 2, 16, seed=18)
    t = list(c.tensors())
    table = t[3].clone()
    table[0, 2], table[0, 7], table[1, 5] = -1, c.nb, 2 ** 30      # holes in one, the last block of the other
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    t[3] = table
    kda_cache_attention(*t, max_new=1, err_flag=err)
    assert err.item() == R.SLOT_RANGE
    got = t[-1].cpu().double().view(2, 4, 128)
    vals = torch.from_numpy(R.e4m3_values())
    for b, n in enumerate(c.lens):
        pos = torch.arange(n)
        blk = table[b].cpu()[pos // 16].long()
        live = (blk >= 0) & (blk < c.nb)
        pos, blk = pos[live], blk[live]
        for h in range(4):
            k = vals[c.k[blk, h // 2, pos % 16].long()] * c.ks[blk, h // 2].double()[:, None]
            v = vals[c.v[blk, h // 2, pos % 16].long()] * c.vs[blk, h // 2].double()[:, None]
            a = torch.softmax(k @ c.q[b].double().view(4, 128)[h] / math.sqrt(128), 0)
            o = a @ v
            assert (got[b, h] - o).abs().max() <= 2.0 ** -6 * (a @ v.abs()).max()
    # a table row that is too narrow for the length
    err.zero_()
    t[3] = t[3][:, :3]
    kda_cache_attention(*t, max_new=1, err_flag=err)
    assert err.item() == R.SLOT_RANGE and not t[-1].isnan().any()


def test_bad_starts_are_skipped(cuda_device):
    c = Case(cuda_device, [50, 60, 70], [2, 1, 2], 4, 2, 16, seed=19)
    t = list(c.tensors())
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    t[1] = torch.tensor([0, 2, 1, 9], dtype=torch.int32, device=cuda_device)   # falls, then passes T
    kda_cache_attention(*t, max_new=2, err_flag=err)
    assert err.item() == R.SEQLENS
    got = t[-1].cpu()
    c.new, c.cu = [2, 0, 0], [0, 2, 2, 2]
    want, tol = c.reference()
    assert ((got[:2].double().view(2, 4, 128) - want[:2]).abs() <= tol[:2]).all() and (got[2:] == 7).all()


def test_max_new_does_not_change_the_result(cuda_device):
    # row tiles of 16, 32 and 64 rows, larger and smaller than the sequences' queries
    # (now 8, 32 and 64 rows, and the variant for prompts)
    c = Case(cuda_device, [300, 200], [5, 2], 12, 2, 16, seed=20)
    for m in (1, 5, 8, 40):
        assert c.check(max_new=m) < 4e-3


def test_large_batches(cuda_device):
    # more sequences than threads in a CTA (the scan over sequences goes in tiles), some without queries
    rng = np.random.default_rng(3)
    lens, new = rng.integers(1, 40, 500).tolist(), rng.integers(0, 2, 500).tolist()
    c = Case(cuda_device, lens, new, 2, 1, 16, seed=21)
    assert c.check() < 4e-3
    c = Case(cuda_device, [1] * 400 + [2000], [1] * 401, 1, 1, 16, seed=22)
    assert c.check() < 4e-3


def test_same_result_every_time_and_a_shared_workspace(cuda_device):
    ws = cache_attention_workspace(48, 8, 4, cuda_device)
    c = Case(cuda_device, [3000, 5000, 10], [4, 4, 4], 48, 8, 64, seed=23)
    d = Case(cuda_device, [900], [3], 48, 8, 64, seed=24)
    t, u = c.tensors(), d.tensors()
    first = None
    for _ in range(20):
        kda_cache_attention(*t, max_new=4, workspace=ws)
        kda_cache_attention(*u, max_new=4, workspace=ws)
        first = t[-1].clone() if first is None else first
        assert torch.equal(first, t[-1])
    c.compare(t[-1])
    d.compare(u[-1])


def test_graphs_that_share_a_workspace_and_new_inputs(cuda_device):
    dev = cuda_device
    ws = cache_attention_workspace(12, 4, 2, dev)
    c, d, e = (Case(dev, lens, [2, 1], 12, 4, 16, seed=s) for lens, s in (([400, 90], 25), ([300, 70], 26), ([390, 20], 27)))
    t, u = c.tensors(), d.tensors()
    calls = [KdaCacheAttentionCall(*x, max_new=2, workspace=ws) for x in (t, u)]
    calls[0]()
    torch.cuda.synchronize(dev)
    graphs = []
    for call in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize(dev)
    c.compare(t[-1])
    d.compare(u[-1])
    # new queries, lengths and pages in the captured buffers
    w = e.tensors()
    for i in (0, 2, 6, 7):
        n = min(t[i].shape[0], w[i].shape[0])
        t[i][:n].copy_(w[i][:n])
    n = min(c.nb, e.nb)
    t[4].view(torch.uint8)[:n].copy_(w[4].view(torch.uint8)[:n])
    t[5].view(torch.uint8)[:n].copy_(w[5].view(torch.uint8)[:n])
    m = min(t[3].shape[1], w[3].shape[1])
    t[3][:, :m].copy_(w[3][:, :m])
    assert e.nb <= c.nb
    graphs[0].replay()
    torch.cuda.synchronize(dev)
    e.compare(t[-1])


def test_other_streams_at_the_same_time(cuda_device):
    # two calls at once, each with a workspace of its own
    dev = cuda_device
    cases = [Case(dev, [2500, 60], [1, 1], 16, 4, 32, seed=30 + i) for i in range(2)]
    ts = [c.tensors() for c in cases]
    calls = [KdaCacheAttentionCall(*t) for t in ts]
    streams = [torch.cuda.Stream(dev) for _ in calls]
    torch.cuda.synchronize(dev)
    for _ in range(10):
        for call, s in zip(calls, streams):
            call(s)
    torch.cuda.synchronize(dev)
    for c, t in zip(cases, ts):
        assert c.compare(t[-1]) < 4e-3


def test_empty_batches(cuda_device):
    c = Case(cuda_device, [5], [0], 4, 2, 16, seed=40, extra=2)
    c.check()
    t = list(c.tensors())
    t[0], t[-1] = t[0][:0], t[-1][:0]
    kda_cache_attention(*t)


def test_refusals(cuda_device):
    c = Case(cuda_device, [50], [2], 4, 2, 16, seed=41)
    t = list(c.tensors())
    kda_cache_attention(*t, max_new=2)

    def refuse(i, bad, **kw):
        u = list(t)
        u[i] = bad
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            kda_cache_attention(*u, max_new=2, **kw)
    refuse(0, t[0].half())
    refuse(0, t[0][:, :500])
    refuse(0, t[0], num_q_heads=3)
    refuse(1, t[1].long())
    refuse(2, t[2].cpu())
    refuse(3, t[3].t())
    refuse(4, t[4].view(torch.uint8))
    refuse(5, t[5][:-1])
    refuse(6, t[6][:, :1])
    refuse(8, t[8][:1])
    refuse(0, t[0], workspace=torch.zeros(100, dtype=torch.int32, device=cuda_device))
    with pytest.raises(ValueError):
        cache_attention_workspace(5, 2, 1, cuda_device)


# The variant for prompts (two groups of 128 rows): chosen by a max_new of more than 96 rows per kv head.
@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("Hq, Hkv", [(1, 1), (6, 2), (24, 3)])
def test_prompt_variant_at_the_edges_of_its_rows(bs, Hq, Hkv, cuda_device):
    # chunks that end below, at and above one group's and both groups' rows, from position 0 and behind cached tokens
    G = Hq // Hkv
    new = sorted({1, 127 // G, 128 // G, 128 // G + 1, 256 // G, 256 // G + 1})
    lens = [n + c for n, c in zip(new, (0, 128, 1, 300, 127, 64, 5))]
    c = Case(cuda_device, lens, new, Hq, Hkv, bs, seed=bs + G, row_pad=8, extra=2)
    assert c.check(max_new=1000) < 4e-3


def test_prompt_variant_joins_parts(cuda_device):
    # one unit over most CTAs (two levels of joins), then some of a few parts each; the same bits every time
    c = Case(cuda_device, [40000], [1], 4, 1, 64, seed=31)
    assert c.check(max_new=1000) < 4e-3
    c = Case(cuda_device, [9000, 3, 4100, 600], [40, 2, 33, 300], 12, 3, 16, seed=32)
    ws = cache_attention_workspace(12, 3, 300, cuda_device)
    t = c.tensors()
    first = None
    for _ in range(4):
        kda_cache_attention(*t, max_new=300, workspace=ws)
        first = t[-1].clone() if first is None else first
        assert torch.equal(first, t[-1])
    assert not ws[:11264].any()
    assert c.compare(t[-1]) < 4e-3


def test_prompt_variant_masks_and_values(cuda_device):
    m = dict(max_new=1000)
    c = Case(cuda_device, [0, 2, 5, 64, 0, 130], [1, 4, 0, 3, 5, 2], 8, 2, 16, seed=7, extra=1)
    c.check(**m)
    c.lens[4] = -3
    c.check(**m)
    c = Case(cuda_device, [700, 300], [2, 1], 8, 2, 16, seed=11)
    g = torch.Generator().manual_seed(1)
    c.vs = torch.exp2(torch.randint(-40, 20, c.vs.shape, generator=g).float())
    c.check(**m)
    c.ks = torch.exp2(torch.randint(-30, 1, c.ks.shape, generator=g).float())
    c.check(**m)
    c = Case(cuda_device, [4096], [1], 4, 1, 16, seed=13, outlier=True)
    c.check(**m)
    c = Case(cuda_device, [20000], [1], 4, 1, 16, seed=14)
    c.k[:] = 0
    c.k[c.table[0, 0].long(), 0, 0] = 0x38
    c.ks[:] = 1.0
    c.q[:] = 1.0
    c.sm = 9.0 / 128
    c.check(**m)
    for scale_q, sm in ((30.0, 0.0), (1.0, -1.0), (1e4, 1e-5), (1e-30, 1e29)):
        c = Case(cuda_device, [300, 129], [1, 3], 12, 4, 32, seed=12, scale_q=scale_q)
        c.sm = sm
        c.check(**m)


@pytest.mark.parametrize("new", [4, 40])
def test_prompt_variant_nan(new, cuda_device):
    # NaN values that the last queries see, that all see; queries and keys that are not finite; in either group of rows
    c = Case(cuda_device, [130, 260], [new, new], 12, 2, 16, seed=9)
    c.v.view(torch.uint8)[c.table[0, 128 // 16].long(), 0, 0, 5] = 0x7f
    c.v.view(torch.uint8)[c.table[0, 128 // 16].long(), 1, 0, 77] = 0xff
    c.v.view(torch.uint8)[c.table[1, 0].long(), 0, 3, 9] = 0x7f
    t = c.tensors()
    t[0][new + 1, 128 * 3 + 7] = float("inf")
    kda_cache_attention(*t, max_new=1000)
    got = t[-1].cpu().double().view(c.T, 2, 6, 128)
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[new - 2:new, 0, :, 5] = True
    nan[new - 2:new, 1, :, 77] = True
    nan[new:, 0, :, 9] = True
    nan[new + 1, 0, 3] = True
    assert torch.equal(got.isnan(), nan)
    c.v = torch.where(c.v & 0x7f == 0x7f, torch.zeros_like(c.v), c.v)
    want, tol = c.reference()
    ok = (got - want.view_as(got)).abs() <= tol.view_as(got)
    assert ok[~nan].all()


def test_prompt_variant_bad_blocks_and_graph(cuda_device):
    c = Case(cuda_device, [200, 90], [3, 40], 4, 2, 16, seed=18)
    t = list(c.tensors())
    want_err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    err = torch.zeros_like(want_err)
    t[3] = t[3].clone()
    t[3][0, 2], t[3][1, 5] = -1, 2 ** 30
    u = list(t)
    u[-1] = t[-1].clone()
    kda_cache_attention(*t, max_new=1, err_flag=want_err)                # the other variant, tested above
    ws = cache_attention_workspace(4, 2, 100, cuda_device)
    call = KdaCacheAttentionCall(*u, max_new=100, err_flag=err, workspace=ws)
    call()
    assert err.item() == want_err.item() == R.SLOT_RANGE
    assert (t[-1].float() - u[-1].float()).norm() <= 2.0 ** -7 * t[-1].float().norm()
    first = u[-1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        u[-1].fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, u[-1])
    assert not ws[:11264].any()


def test_prompt_variant_batches_and_heads(cuda_device):
    # more sequences than threads, most without queries; more heads per kv head than a tile has rows
    rng = np.random.default_rng(4)
    lens, new = rng.integers(1, 40, 900).tolist(), rng.integers(0, 2, 900).tolist()
    c = Case(cuda_device, lens, new, 2, 1, 16, seed=33)
    assert c.check(max_new=100) < 4e-3
    for Hq in (130, 300):
        c = Case(cuda_device, [150, 40, 9], [2, 1, 3], Hq, 1, 32, seed=Hq)
        assert c.check(max_new=3) < 4e-3
        assert c.check(max_new=1) < 4e-3


def test_both_kernels_share_a_workspace_and_run_side_by_side(cuda_device):
    ws = cache_attention_workspace(12, 2, 300, cuda_device)
    c = Case(cuda_device, [3000, 700, 10], [60, 200, 4], 12, 2, 64, seed=34)
    d = Case(cuda_device, [9000, 500], [1, 2], 12, 2, 64, seed=35)
    t, u = c.tensors(), d.tensors()
    for _ in range(3):                                      # one after the other, the same workspace
        kda_cache_attention(*t, max_new=300, workspace=ws)
        kda_cache_attention(*u, max_new=2, workspace=ws)
    assert c.compare(t[-1]) < 4e-3 and d.compare(u[-1]) < 4e-3
    first, second = t[-1].clone(), u[-1].clone()
    side = torch.cuda.Stream()
    a, b = KdaCacheAttentionCall(*t, max_new=300), KdaCacheAttentionCall(*u, max_new=2)
    again = KdaCacheAttentionCall(*t[:-1], torch.empty_like(first), max_new=300)
    for _ in range(10):                                     # at the same time, a workspace each
        a()
        with torch.cuda.stream(side):
            b(side)
            again(side)
    torch.cuda.synchronize()
    assert torch.equal(first, t[-1]) and torch.equal(second, u[-1]) and torch.equal(first, again._keep[8])


COUNTERS = 45056 // 4        # KDA_CACHE_ATTENTION_COUNTER_BYTES
# (query heads, kv heads, queries): 8, 16, 24, 32, 64 and 96 query rows per kv head, one variant each, and 120 for prompts
VARIANTS = [(4, 2, 4), (8, 2, 4), (12, 2, 4), (16, 2, 4), (32, 2, 4), (24, 1, 4), (48, 2, 5)]


@pytest.mark.parametrize("Hq, Hkv, new", VARIANTS)
def test_every_row_tile_joins_many_parts(Hq, Hkv, new, cuda_device):
    # units over more than eight CTAs (two levels of joins) beside short ones; the same bits every time, whichever part
    # comes last, and the whole counter area is zero again
    c = Case(cuda_device, [20000, 5, 2500], [new] * 3, Hq, Hkv, 64, seed=50 + Hq)
    ws = cache_attention_workspace(Hq, Hkv, new, cuda_device)
    t = c.tensors()
    first = None
    for _ in range(20):
        t[-1].fill_(7.0)
        kda_cache_attention(*t, max_new=new, workspace=ws)
        first = t[-1].clone() if first is None else first
        assert torch.equal(first, t[-1])
        assert not ws[:COUNTERS].any()
    assert c.compare(t[-1]) < 4e-3


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("Hq, Hkv, new", [(8, 1, 1), (6, 2, 5), (20, 2, 2), (10, 2, 5), (16, 2, 4), (11, 1, 3), (16, 2, 8),
                                          (13, 1, 5), (24, 2, 8), (97, 1, 1)])
def test_every_row_tile_at_every_block_size(bs, Hq, Hkv, new, cuda_device):
    # 8, 15, 20, 25, 32, 33, 64, 65, 96 and 97 query rows per kv head: both ends of every variant's range, whose block
    # scales and copies differ with the block size; lengths around a tile, several tiles, parts of several CTAs
    lens = [max(n, new) for n in (new, 127, 128, 129, 1, 300, 3000)]
    c = Case(cuda_device, lens, [new] * len(lens), Hq, Hkv, bs, seed=bs + Hq + new, row_pad=8, extra=2)
    ws = cache_attention_workspace(Hq, Hkv, new, cuda_device)
    assert c.check(ws=ws) < 4e-3
    assert not ws[:COUNTERS].any()


@pytest.mark.parametrize("bs", [16, 128, 256])
@pytest.mark.parametrize("Hq, Hkv, new", VARIANTS)
def test_every_row_tile_masks_and_values(Hq, Hkv, new, bs, cuda_device):
    # rows that see nothing, lengths of zero and below the queries; values that are not finite and that the last query
    # alone, or all queries, see; a key that is NaN and only the last query sees; an infinite query
    c = Case(cuda_device, [0, new - 2, new, 300, 133], [new] * 5, Hq, Hkv, bs, seed=70 + Hq + bs, extra=1)
    c.check()
    last = Hkv - 1
    c.v[c.table[3, 299 // bs].long(), 0, 299 % bs, 5] = 0x7f                  # position 299 of 300: the last query's own
    c.v[c.table[4, 2 // bs].long(), last, 2 % bs, 9] = 0xff                   # position 2: every query of the sequence
    c.k[c.table[4, 132 // bs].long(), 0, 132 % bs, 8] = 0x7f                  # the last token of 133
    c.q[3 * new, 128 * (Hq - 1) + 3] = float("inf")                           # first query, last head of the fourth
    t = c.tensors()
    kda_cache_attention(*t, max_new=new)
    got = t[-1].cpu().double().view(c.T, Hkv, Hq // Hkv, 128)
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[4 * new - 1, 0, :, 5] = True
    nan[4 * new:5 * new, last, :, 9] = True
    nan[5 * new - 1, 0] = True
    nan[3 * new, last, -1] = True
    assert torch.equal(got.isnan(), nan)
    # all else is as if the values and the key were finite
    c.v = torch.where(c.v & 0x7f == 0x7f, torch.zeros_like(c.v), c.v)
    c.k = torch.where(c.k & 0x7f == 0x7f, torch.zeros_like(c.k), c.k)
    c.q[3 * new, 128 * (Hq - 1) + 3] = 0.0
    want, tol = c.reference()
    ok = (got - want.view_as(got)).abs() <= tol.view_as(got)
    assert ok[:c.cu[-1]][~nan[:c.cu[-1]]].all()
