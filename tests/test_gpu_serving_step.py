"""The serving-step operators together, as a speculative serving loop uses
them: block tables from the lengths, norm + rotation + cache write and
attention of a softmax layer, the multi-token step of a KDA layer, and the
verification that decides how far every sequence got, whose state slot the
next step starts from and how many tokens its cache keeps.  The whole step
is one CUDA graph; between replays only lengths, slots and inputs change, all
on the device."""
import math

import numpy as np
import pytest
import torch

import step_reference as R
from linear_attention_decode_04_gb300 import (KdaBlockTablesCall, KdaCacheAttentionCall, KdaDecodeCall, KdaQkRopeCall,
                                              KdaVerifyDraftCall, rope_frequencies)
from linear_attention_decode_04_gb300.stack import warm_up

pytestmark = pytest.mark.gpu

N, T, HQ, HKV, BS, V, KH = 5, 3, 6, 2, 16, 211, 2
BASE = 1e4


class Loop:
    """Buffers and captured step; sequence N - 1 is padding (no tokens, source slot 0)."""

    def __init__(self, dev):
        self.dev = dev
        g = torch.Generator().manual_seed(0)
        f = lambda *s, sc=1.0: (torch.randn(*s, generator=g) * sc).to(dev)  # noqa: E731
        i = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        R_ = N * T
        self.cached, self.held = i([13, 0, 30, 16, 0]), i([1, 0, 2, 1, 0])
        self.new = i([T] * (N - 1) + [0])
        self.blocks = 40
        self.table = torch.full((N, 8), -1, dtype=torch.int32, device=dev)
        self.table[0, :1], self.table[2, :2], self.table[3, :1] = i([7]), i([30, 2]), i([11])
        self.free = i([b for b in np.random.default_rng(1).permutation(40).tolist() if b not in (7, 30, 2, 11)])
        self.head = i([0])
        self.err = i([0])
        self.tables = KdaBlockTablesCall(self.cached, self.new, self.table, self.free, self.head, block_size=BS,
                                         num_blocks=self.blocks, num_tokens=R_, held_blocks=self.held, err_flag=self.err)
        # softmax layer
        self.qkv = f(R_, (HQ + 2 * HKV) * 128).bfloat16()
        self.q = torch.empty(R_, HQ * 128, dtype=torch.bfloat16, device=dev)
        self.wq, self.wk = 1 + f(128, sc=0.1), 1 + f(128, sc=0.1)
        shape = (self.blocks, HKV, BS, 128)
        # what the cache held before: tokens that this test's bookkeeping does not know count through the cache itself
        self.kc, self.vc = ((torch.randn(shape, generator=g) * 60).clamp(-440, 440).to(torch.float8_e4m3fn).to(dev)
                            for _ in range(2))
        self.ks, self.vs = (torch.full((self.blocks, HKV), 2.0 ** -6, device=dev) for _ in range(2))
        self.rope = KdaQkRopeCall(self.qkv, self.tables.positions, self.q, num_q_heads=HQ, num_kv_heads=HKV,
                                  rope_freqs=rope_frequencies(64, BASE, dev), q_weight=self.wq, k_weight=self.wk,
                                  k_cache=self.kc, v_cache=self.vc, k_scale=self.ks, v_scale=self.vs,
                                  slot_map=self.tables.slot_map, err_flag=self.err)
        self.out = torch.full((R_, HQ * 128), 3.0, dtype=torch.bfloat16, device=dev)
        self.attn = KdaCacheAttentionCall(self.q, self.tables.cu_seqlens, self.tables.seq_lens, self.table, self.kc,
                                          self.vc, self.ks, self.vs, self.out, max_new=T, err_flag=self.err)
        # KDA layer: slots 1 .. N*(T+1), every sequence with T + 1 of its own
        D = KH * 128
        slots = N * (T + 1) + 1
        self.state, self.conv = f(slots, KH, 128, 128, sc=0.02), f(slots, 3 * D, 3).bfloat16()
        self.src = i([1 + n * (T + 1) for n in range(N - 1)] + [0])
        self.dst = i([[2 + n * (T + 1) + t for t in range(T)] for n in range(N)])
        self.kout = torch.empty(R_, D, dtype=torch.bfloat16, device=dev)
        self.kda_in = dict(qkv=f(R_, 3 * D).bfloat16(), g=-torch.rand(R_, KH, 128, generator=g).to(dev),
                           beta=torch.rand(R_, KH, generator=g).to(dev).bfloat16(), gate=f(R_, D).bfloat16())
        self.kda = KdaDecodeCall(self.kda_in["qkv"], f(3, 4, D, sc=0.5), self.conv, self.state, self.kda_in["g"],
                                 self.kda_in["beta"], self.dst, self.kout, gate=self.kda_in["gate"],
                                 norm_weight=1 + f(128, sc=0.1), tokens_per_seq=T, src_slot=self.src, err_flag=self.err)
        # verification
        self.draft = torch.zeros(N, T - 1, dtype=torch.int32, device=dev)
        self.p, self.dp = torch.zeros(N, T, V, device=dev), torch.zeros(N, T - 1, V, device=dev)
        self.u, self.su = torch.zeros(N, T - 1, device=dev), torch.zeros(N, device=dev)
        self.verify = KdaVerifyDraftCall(self.draft, self.p, self.u, self.su, draft_probs=self.dp, src_slot=self.src,
                                         slot_idx=self.dst, err_flag=self.err)

    def step(self):
        self.tables()
        self.rope()
        self.attn()
        self.kda()
        self.verify()

    def advance(self):
        """The next step's lengths, blocks and slots, on the device: the slot that the step ended in becomes the
        source, and the old source takes its place among the destinations."""
        active = self.src > 0
        self.cached.add_(torch.where(active, self.verify.num_accepted + 1, torch.zeros_like(self.cached)))
        self.held.copy_(self.tables.held_blocks_out)
        self.head.copy_(self.tables.free_head_out)
        took = self.dst == self.verify.next_slot[:, None]
        self.dst.copy_(torch.where(took & active[:, None], self.src[:, None], self.dst))
        self.src.copy_(self.verify.next_slot)


def test_speculative_serving_loop(cuda_device):
    dev = cuda_device
    warm_up(dev)
    L = Loop(dev)
    torch.cuda.synchronize(dev)
    # one eager step on a copy of nothing in particular loads every kernel before the capture; its effects are undone
    keep = {k: getattr(L, k).clone() for k in ("table", "ks", "vs", "state", "conv")}
    codes = [c.view(torch.uint8).clone() for c in (L.kc, L.vc)]
    L.step()
    torch.cuda.synchronize(dev)
    for k, v in keep.items():
        getattr(L, k).copy_(v)
    for c, v in zip((L.kc, L.vc), codes):
        c.view(torch.uint8).copy_(v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.step()
        L.advance()
    rng = np.random.default_rng(9)
    vals = torch.from_numpy(R.e4m3_values())
    freqs = R.inv_freqs(64, BASE)
    head, held = 0, L.held.tolist()
    accepted_all = []
    for step in range(12):
        # new token inputs, drafts and random numbers
        for t in (L.qkv, L.kda_in["qkv"], L.kda_in["gate"]):
            t.copy_(torch.from_numpy(rng.normal(size=tuple(t.shape)).astype(np.float32)))
        z = rng.normal(size=(N, T, V)) * 2
        p = np.exp(z) / np.exp(z).sum(-1, keepdims=True)
        q = np.exp(z[:, :-1] + rng.normal(size=(N, T - 1, V)) * 0.7)
        q /= q.sum(-1, keepdims=True)
        p, q = p.astype(np.float32), q.astype(np.float32)
        d = np.array([[rng.choice(V, p=q[n, t] / q[n, t].astype(np.float64).sum()) for t in range(T - 1)]
                      for n in range(N)], np.int32)
        u, su = rng.random((N, T - 1), np.float32), rng.random(N, np.float32)
        for dst, src in ((L.p, p), (L.dp, q), (L.draft, d), (L.u, u), (L.su, su)):
            dst.copy_(torch.from_numpy(src))
        before = dict(cached=L.cached.tolist(), table=L.table.cpu().numpy(), src=L.src.tolist(), dst=L.dst.tolist())
        # the KDA layer's own result on the same inputs, by single-token steps: states after every token
        state, conv = L.state.clone(), L.conv.clone()
        graph.replay()
        torch.cuda.synchronize(dev)
        assert L.err.item() == 0
        # ---- metadata
        want = R.block_tables(before["cached"], [T] * (N - 1) + [0], before["table"], L.free.tolist(), head, BS,
                              L.blocks, N * T, held)
        assert np.array_equal(L.table.cpu().numpy(), want[0])
        assert L.tables.slot_map.tolist() == want[4] and L.tables.positions.tolist() == want[3]
        head, held = want[5], want[6]
        assert L.head.item() == head and L.held.tolist() == held
        # ---- the cache holds this step's keys and values at their positions
        x = L.qkv.cpu().double().numpy().reshape(N * T, HQ + 2 * HKV, 128)
        kc, vc = (vals[c.view(torch.uint8).cpu().long()] * s.cpu().double()[..., None, None]
                  for c, s in ((L.kc, L.ks), (L.vc, L.vs)))
        for r in range((N - 1) * T):
            b, o = divmod(want[4][r], BS)
            k = R.norm_rotate(x[r, HQ:HQ + HKV], L.wk.cpu().numpy(), want[3][r], freqs, False, 1e-6)
            for got, exact, s in ((kc[b, :, o], k, L.ks[b]), (vc[b, :, o], x[r, HQ + HKV:], L.vs[b])):
                lim = np.maximum(2.0 ** -4 * np.abs(exact), 2.0 ** -10 * s.cpu().numpy()[:, None]) + 2.0 ** -19 * 16
                # (rows of blocks whose scale grew later in the same run are rounded once, so this bound is enough)
                assert (np.abs(got.numpy() - exact) <= lim).all(), (step, r)
        # ---- attention over what the cache holds
        qn = L.q.cpu().double().view(N * T, HQ, 128)
        got = L.out.cpu().double().view(N * T, HQ, 128)
        for r in range((N - 1) * T):
            n, pos = divmod(r, T)[0], want[3][r]
            at = [(want[0][n][s // BS], s % BS) for s in range(pos + 1)]
            blk, off = torch.tensor([a for a, _ in at]), torch.tensor([b for _, b in at])
            for h in range(HQ):
                kk, vv = kc[blk, h // (HQ // HKV), off], vc[blk, h // (HQ // HKV), off]
                a = torch.softmax(kk @ qn[r, h] / math.sqrt(128), 0)
                tol = 2.0 ** -8 * (a @ vv).abs() + (2.0 ** -8 + 2.0 ** -9) * (a @ vv.abs()) + 2.0 ** -9 * (a[:, None] * vv.abs()).max()
                assert ((got[r, h] - a @ vv).abs() <= tol + 1e-9).all(), (step, r, h)
        assert (got[(N - 1) * T:] == 3.0).all()          # the padding sequence's rows are left as they were
        # ---- verification, and the slot that the next step starts from
        tok, acc, nxt, _ = R.verify(d, p, u, su, q, before["src"], before["dst"])
        assert L.verify.tokens.tolist() == tok and L.verify.num_accepted.tolist() == acc
        assert L.src.tolist() == nxt
        accepted_all += acc[:-1]
        assert L.cached.tolist() == [c + a + 1 if s > 0 else c for c, a, s in zip(before["cached"], acc, before["src"])]
        # ---- the state in that slot is that of the accepted tokens alone
        for n in range(N - 1):
            one = KdaDecodeCall(L.kda_in["qkv"][n * T:n * T + acc[n] + 1].contiguous(), L.kda._keep[1], conv, state,
                                L.kda_in["g"][n * T:n * T + acc[n] + 1].contiguous(),
                                L.kda_in["beta"][n * T:n * T + acc[n] + 1].contiguous(),
                                torch.tensor([before["dst"][n][:acc[n] + 1]], dtype=torch.int32, device=dev),
                                torch.empty(acc[n] + 1, KH * 128, dtype=torch.bfloat16, device=dev),
                                gate=L.kda_in["gate"][n * T:n * T + acc[n] + 1].contiguous(), norm_weight=L.kda._keep[9],
                                tokens_per_seq=acc[n] + 1,
                                src_slot=torch.tensor([before["src"][n]], dtype=torch.int32, device=dev))
            one()
            torch.cuda.synchronize(dev)
            assert torch.equal(L.conv[nxt[n]], conv[nxt[n]])
            assert (L.state[nxt[n]] - state[nxt[n]]).abs().max() <= 1e-4
    assert {0, 1, 2} <= set(accepted_all)                # every outcome was met
