"""The operators between and behind the layers together with a KDA layer and the
verification, as a speculative serving step uses them: the residual's norm
feeds an 8-bit projection that makes the layer's q, k, v; the layer's output is
made 8-bit and projected back onto the residual stream; a gated feed-forward
block does the same; the head's logits are verified and reported.  The whole
step is one CUDA graph that runs several times, each operator checked against
64 bits on what it was given."""
import pytest
import torch

import layer_reference as R
from linear_attention_decode_04_gb300 import (KdaAddNormCall, KdaDecodeCall, KdaLinearCall, KdaLogprobsCall,
                                              KdaVerifyDraftCall)
from linear_attention_decode_04_gb300.stack import warm_up
from test_gpu_step_streams import results_in_used_memory

pytestmark = pytest.mark.gpu

N, T, H, D, F, V = 3, 3, 2, 320, 416, 1003       # sequences, tokens of a step, heads, width, feed-forward width, vocabulary
ROWS, HD = N * T, 128 * H
F8 = torch.float8_e4m3fn
INNER = 2.0 ** -18                               # of fp32 arithmetic inside the norm (see its own tests)


class Step:
    def __init__(self, dev):
        g = torch.Generator().manual_seed(0)
        f = lambda *s, sc=1.0: (torch.randn(*s, generator=g) * sc).to(dev)  # noqa: E731
        b16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
        i = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731

        def weights8(n, k):
            w = f(n, k) / k ** 0.5
            s = w.abs().amax(-1) / 448
            return (w / s[:, None]).to(F8), s

        def codes(d):
            return torch.zeros(ROWS, d, device=dev).to(F8), torch.zeros(ROWS, device=dev)
        self.err = i([0])
        self.stream = f(ROWS, D, sc=2.0).bfloat16()                 # the residual stream, in place
        self.layer_in = f(ROWS, D).bfloat16()                       # what the layer ahead gave
        self.w_norm = [1 + f(D, sc=0.1) for _ in range(3)]
        self.q1, self.s1 = codes(D)
        self.norm1 = KdaAddNormCall(self.layer_in, weight=self.w_norm[0], residual=self.stream, residual_out=self.stream,
                                    out_q=self.q1, out_scale=self.s1)
        self.w_qkv, self.ws_qkv = weights8(3 * HD, D)
        self.qkv = b16(ROWS, 3 * HD)
        self.to_qkv = KdaLinearCall(self.q1, self.w_qkv, self.qkv, x_scale=self.s1, weight_scale=self.ws_qkv, early_weight=True,
                                    err_flag=self.err)
        slots = 1 + N * (T + 1)
        self.state, self.conv = f(slots, H, 128, 128, sc=0.02), f(slots, 3 * HD, 3).bfloat16()
        self.src = i([1 + n * (T + 1) for n in range(N)])
        self.dst = i([[2 + n * (T + 1) + t for t in range(T)] for n in range(N)])
        self.kda_out = b16(ROWS, HD)
        self.kda = KdaDecodeCall(self.qkv, f(3, 4, HD, sc=0.5), self.conv, self.state,
                                 -torch.rand(ROWS, H, 128, generator=g).to(dev), torch.rand(ROWS, H, generator=g).to(dev).bfloat16(),
                                 self.dst, self.kda_out, gate=f(ROWS, HD).bfloat16(), norm_weight=1 + f(128, sc=0.1),
                                 tokens_per_seq=T, src_slot=self.src, err_flag=self.err)
        self.q2, self.s2 = codes(HD)
        self.quantise = KdaAddNormCall(self.kda_out, out_q=self.q2, out_scale=self.s2, norm=False)
        self.w_out, self.ws_out = weights8(D, HD)
        self.from_kda = KdaLinearCall(self.q2, self.w_out, self.stream, x_scale=self.s2, weight_scale=self.ws_out,
                                      residual=self.stream, early_weight=True, err_flag=self.err)
        self.y2 = b16(ROWS, D)
        self.norm2 = KdaAddNormCall(self.stream, weight=self.w_norm[1], out=self.y2)
        self.w_up = f(2 * F, D, sc=D ** -0.5).bfloat16()
        self.up = b16(ROWS, F)
        self.gated = KdaLinearCall(self.y2, self.w_up, self.up, activation="silu_gated", early_weight=True, err_flag=self.err)
        self.w_down = f(D, F, sc=F ** -0.5).bfloat16()
        self.mlp = b16(ROWS, D)
        self.down = KdaLinearCall(self.up, self.w_down, self.mlp, early_weight=True, err_flag=self.err)
        self.y3 = b16(ROWS, D)
        self.norm3 = KdaAddNormCall(self.mlp, weight=self.w_norm[2], residual=self.stream, residual_out=self.stream, out=self.y3)
        self.w_head = f(V, D, sc=3 * D ** -0.5).bfloat16()
        self.logits = torch.empty(ROWS, V, device=dev)
        self.head = KdaLinearCall(self.y3, self.w_head, self.logits, early_weight=True, err_flag=self.err)
        self.probs = torch.empty(N, T, V, device=dev)
        self.draft = torch.zeros(N, T - 1, dtype=torch.int32, device=dev)
        self.u, self.su = torch.zeros(N, T - 1, device=dev), torch.zeros(N, device=dev)
        self.verify = KdaVerifyDraftCall(self.draft, self.probs, self.u, self.su, src_slot=self.src, slot_idx=self.dst,
                                         err_flag=self.err)
        self.report = KdaLogprobsCall(self.logits.view(N, T, V), self.verify.tokens, num_top=4, err_flag=self.err)

    def run(self, keep=None):
        """One step; with ``keep``, the residual stream as each operator finds it."""
        see = (lambda name: keep.__setitem__(name, self.stream.clone())) if keep is not None else lambda name: None
        see("0")
        self.norm1()
        see("1")
        self.to_qkv(), self.kda(), self.quantise(), self.from_kda()
        see("2")
        self.norm2(), self.gated(), self.down(), self.norm3()
        see("3")
        self.head()
        self.probs.copy_(torch.softmax(self.logits, -1).view(N, T, V))
        self.verify(), self.report()


def close(got, want, tol, bf16=True):
    d = (got.cpu().double() - want).abs()
    assert (d <= tol + (want.abs() + tol) * (R.BF16 if bf16 else 0) + 1e-30).all(), d.max()


def check(s, keep):
    c = lambda t: t.cpu()  # noqa: E731

    def normed(x, w, residual, out, codes=None, norm=True):
        h, y, sc = R.add_norm(c(x), None if w is None else c(w), None if residual is None else c(residual), norm=norm)
        if out is not None:
            close(out, y, y.abs() * INNER)
        if codes is not None:
            q, scale = c(codes[0]).double(), c(codes[1]).double()
            assert ((scale - sc).abs() <= sc * INNER).all()
            v = y / sc[:, None]
            assert ((q - v).abs() <= v.abs() * (R.E4M3 + INNER) + R.E4M3_TINY).all()
        return h

    def product(x, w, out, bf16=True, **kw):
        want, tol = R.linear(c(x), c(w), **{k: c(v) if isinstance(v, torch.Tensor) else v for k, v in kw.items()})
        close(out, want, tol, bf16)
    h = normed(s.layer_in, s.w_norm[0], keep["0"], None, (s.q1, s.s1))
    close(keep["1"], h, h.abs() * R.FP32)
    product(s.q1, s.w_qkv, s.qkv, x_scale=s.s1, weight_scale=s.ws_qkv)
    normed(s.kda_out, None, None, None, (s.q2, s.s2), norm=False)
    product(s.q2, s.w_out, keep["2"], x_scale=s.s2, weight_scale=s.ws_out, residual=keep["1"])
    normed(keep["2"], s.w_norm[1], None, s.y2)
    product(s.y2, s.w_up, s.up, activation="silu_gated")
    product(s.up, s.w_down, s.mlp)
    h = normed(s.mlp, s.w_norm[2], keep["2"], s.y3)
    close(keep["3"], h, h.abs() * R.FP32)
    product(s.y3, s.w_head, s.logits, False)
    tokens = c(s.verify.tokens)
    assert ((tokens >= 0).sum(1) == c(s.verify.num_accepted) + 1).all()     # the drafts that stand, and one more
    lp, ranks, ent, ids, top, scale = R.logprobs(c(s.logits).view(N, T, V), tokens, 4)
    assert torch.equal(c(s.report.ranks), ranks) and torch.equal(c(s.report.top_ids), ids)
    for got, want, tol in ((s.report.logprobs, lp, 2.0 ** -17 + lp.abs() * 2.0 ** -22), (s.report.entropy, ent, 2.0 ** -17 * scale),
                           (s.report.top_logprobs, top, 2.0 ** -17 + top.abs() * 2.0 ** -22)):
        assert ((c(got).double() - want).abs() <= tol).all()
    assert s.err.item() == 0


def test_speculative_step(cuda_device):
    dev = cuda_device
    warm_up(dev)
    s = Step(dev)
    rng = torch.Generator().manual_seed(5)

    def new_inputs():
        s.layer_in.copy_(torch.randn(ROWS, D, generator=rng))
        s.stream.copy_(torch.randn(ROWS, D, generator=rng) * 2)
        s.draft.copy_(torch.randint(0, V, (N, T - 1), generator=rng))
        s.u.copy_(torch.rand(N, T - 1, generator=rng) * 1e-3)
        s.su.copy_(torch.rand(N, generator=rng))
    new_inputs()
    keep = {}
    s.run(keep)                                        # eagerly, which loads every kernel too
    torch.cuda.synchronize(dev)
    check(s, keep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        keep = {}
        s.run(keep)
    for _ in range(4):
        new_inputs()
        state, conv = s.state.clone(), s.conv.clone()
        graph.replay()
        torch.cuda.synchronize(dev)
        check(s, keep)
        # the layer itself: the same call alone, from the same state
        out = s.kda_out.clone()
        after = s.state.clone()
        s.state.copy_(state), s.conv.copy_(conv)
        s.kda()
        torch.cuda.synchronize(dev)
        assert torch.equal(out, s.kda_out) and torch.equal(after, s.state)


def test_report_in_used_memory(cuda_device):
    # results that went into memory which work on the stream they were made on still writes
    g = torch.Generator().manual_seed(1)
    x, t = torch.randn(5, 700, generator=g), torch.randint(0, 700, (5,), generator=g, dtype=torch.int32)
    gx, gt = x.to(cuda_device), t.to(cuda_device)
    call = results_in_used_memory(lambda: KdaLogprobsCall(gx, gt, num_top=3), lambda c: (c.logprobs, c.ranks, c.entropy, c.top_ids))
    want = R.logprobs(x, t, 3)
    assert torch.equal(call.ranks.cpu(), want[1]) and torch.equal(call.top_ids.cpu(), want[3])


def test_two_streams_at_once(cuda_device):
    # calls without workspaces: two of each kind side by side, on tensors of their own
    dev = cuda_device
    g = torch.Generator().manual_seed(2)
    x = [torch.randn(200, 512, generator=g).bfloat16() for _ in range(2)]
    w = [torch.randn(700, 512, generator=g).bfloat16() for _ in range(2)]
    gx, gw = [t.to(dev) for t in x], [t.to(dev) for t in w]
    alone = []
    for i in range(2):
        y, z = torch.empty_like(gx[i]), torch.empty(200, 700, device=dev)
        calls = [KdaAddNormCall(gx[i], out=y), KdaLinearCall(y, gw[i], z), KdaLogprobsCall(z, num_top=8)]
        for c in calls:
            c()
        torch.cuda.synchronize(dev)
        alone.append((calls, y, z, [v.clone() for v in (y, z, calls[2].entropy, calls[2].top_ids)]))
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    for calls, y, z, _ in alone:
        y.zero_(), z.zero_()
    for st in streams:
        st.wait_stream(torch.cuda.current_stream(dev))
    for _ in range(30):
        for st, (calls, *_r) in zip(streams, alone):
            for c in calls:
                c(st)
    torch.cuda.synchronize(dev)
    for calls, y, z, want in alone:
        for a, b in zip((y, z, calls[2].entropy, calls[2].top_ids), want):
            assert torch.equal(a, b)
