"""Log probabilities, ranks, entropy and top alternatives against 64 bits: whole
numbers have to be equal."""
import math

import pytest
import torch

import layer_reference as R
from linear_attention_decode_04_gb300 import KdaLogprobsCall, kda_logprobs

pytestmark = pytest.mark.gpu

# a thread adds at most 64 terms one after another and a row's sums meet in 12 steps; the exponential is off by 2^-21,
# the logarithm by 2^-23: below 2^-17, times what the quantity is made of
INNER = 2.0 ** -17


def same(got, want, tol):
    got = got.cpu().double()
    want = torch.where(want.abs() > 3.4028235677973366e38, want.sign() * math.inf, want)   # (what fp32 rounds to infinity)
    assert torch.equal(got.isnan(), want.isnan())
    inf = want.abs() == math.inf
    assert torch.equal(got[inf], want[inf])
    ok = ~(want.isnan() | inf)
    assert ((got - want).abs()[ok] <= tol.expand_as(want)[ok]).all(), ((got - want).abs()[ok].max())


def check(dev, logits, tokens=None, num_top=0, gpu_logits=None, err=0):
    flag = torch.zeros(1, dtype=torch.int32, device=dev)
    got = kda_logprobs(logits.to(dev) if gpu_logits is None else gpu_logits, None if tokens is None else tokens.to(dev),
                       num_top=num_top, err_flag=flag)
    lp, ranks, ent, ids, top, scale = R.logprobs(logits, tokens, num_top)
    assert flag.item() == err
    if tokens is None:
        assert got[0] is None and got[1] is None
    else:
        assert torch.equal(got[1].cpu(), ranks)
        same(got[0], lp, INNER + lp.abs() * 2.0 ** -22)
    same(got[2], ent, INNER * scale)
    assert torch.equal(got[3].cpu(), ids)
    same(got[4], top, INNER + top.abs() * 2.0 ** -22)
    return got


def rows(R_, V, seed, dt=torch.float32, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(R_, V, generator=g) * spread).to(dt)
    return x, torch.randint(0, V, (R_,), generator=g, dtype=torch.int32)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R_, V, k", [(1, 1, 1), (2, 2, 5), (3, 31, 32), (4, 300, 20), (5, 1000, 32), (2, 4096, 7), (7, 4099, 32),
                                      (1, 131072, 20), (3, 100003, 5), (33, 32001, 8), (90, 5003, 32), (160, 20011, 3),
                                      (400, 1027, 20), (700, 2048, 1), (1300, 129, 0)])
def test_matches_64_bits(R_, V, k, dt, cuda_device):
    x, t = rows(R_, V, R_ + V, dt)
    check(cuda_device, x, t, k)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 7])
def test_rows_on_any_boundary(offset, dt, cuda_device):
    x, t = rows(6, 3001, offset, dt)
    wide = torch.full((6, 3001 + 16), 50.0, dtype=dt, device=cuda_device)    # larger than everything in the rows
    view = wide[:, offset:offset + 3001]
    view.copy_(x)
    check(cuda_device, x, t, 9, gpu_logits=view)


@pytest.mark.parametrize("V", [7, 300, 5000, 70001])
@pytest.mark.parametrize("kind", ["rising", "falling", "equal", "two values", "steps", "zeros"])
def test_orders_and_ties(kind, V, cuda_device):
    i = torch.arange(V, dtype=torch.float32)
    x = {"rising": i / V, "falling": -i / V, "equal": torch.full((V,), -1.25), "two values": (i % 3 == 1).float(),
         "steps": torch.floor(i / 40) % 50, "zeros": torch.where(i % 2 == 0, -0.0, 0.0)}[kind]
    x = torch.stack([x, x.flip(0)])
    for tok in (0, V // 2, V - 1):
        check(cuda_device, x, torch.tensor([tok, tok], dtype=torch.int32), 32)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R_, V, k", [(20, 1416, 27), (49, 415, 27), (549, 424, 7), (700, 255, 32), (700, 4097, 32), (620, 8192, 20),
                                      (620, 8200, 20), (1900, 1030, 32), (1900, 5001, 9)])
def test_short_rows(R_, V, k, dt, cuda_device):
    # fewer vectors than threads, fewer threads with any than alternatives; small CTAs and large ones
    x, t = rows(R_, V, R_ * V, dt)
    check(cuda_device, x, t, k)


@pytest.mark.parametrize("V", [9, 130, 600, 5000])
@pytest.mark.parametrize("kind", ["rising", "equal", "steps", "ruled out"])
def test_orders_and_ties_in_many_rows(kind, V, cuda_device):
    i = torch.arange(V, dtype=torch.float32)
    x = {"rising": i / V, "equal": torch.full((V,), 3.0), "steps": torch.floor(i / 40) % 5,
         "ruled out": torch.where(i % 97 == 8, i / 64, -math.inf)}[kind].repeat(640, 1)
    check(cuda_device, x, torch.arange(640, dtype=torch.int32) % V, 32)


@pytest.mark.parametrize("rows_", [1, 3, 700])
def test_large_logits_in_one_threads_elements(rows_, cuda_device):
    # the largest elements all in places that one thread, or few, go through
    V = 60000
    x, t = rows(rows_, V, 5)
    x[:, 8::1024] += 100.0
    x[:, 9::1024] += 90.0
    check(cuda_device, x, t, 32)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows_, V", [(2, 700), (2, 5003), (3, 40001), (1, 300007), (700, 1030), (640, 9001)])
def test_many_equal_elements_at_the_bound(rows_, V, dt, cuda_device):
    # more of them than a CTA lists, behind few that are larger: the first of them, wherever they begin
    i = torch.arange(V)
    few = torch.zeros(V)
    few[[V - 1, V // 2, 3]] = torch.tensor([2.0, 1.0, 2.0])
    low = torch.full((V,), -8.0)
    kinds = [few, torch.where(i >= V - V // 3, 0.0, low), torch.where(i < V // 3, 0.0, low) + 4 * few, torch.where(i % 5 == 2, 0.0, low),
             torch.where(i >= V - 40, 0.0, low), torch.where(i % 2 == 0, -math.inf, 0.0) + few]
    for k, x in enumerate(kinds):
        x = x.repeat(rows_, 1).to(dt)
        wide = torch.full((rows_, V + 13), 50.0, dtype=dt, device=cuda_device)[:, k:k + V]
        wide.copy_(x)
        check(cuda_device, x, torch.full((rows_,), V - 1, dtype=torch.int32), 32, gpu_logits=wide)


@pytest.mark.parametrize("R_, V, dt", [(256, 131072, torch.float32), (1000, 100003, torch.bfloat16)])
def test_rows_of_one_value_take_no_longer_than_a_few_others(R_, V, dt, cuda_device):
    g = torch.Generator(device=cuda_device).manual_seed(0)
    t = torch.zeros(R_, dtype=torch.int32, device=cuda_device)

    def time(x):
        call = KdaLogprobsCall(x.to(dt), t, num_top=20)
        best = math.inf
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(4):
                call()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    usual = time(torch.randn(R_, V, generator=g, device=cuda_device) * 3)
    for v in (0.0, math.nan, math.inf, -math.inf):
        assert time(torch.full((R_, V), v, device=cuda_device)) < 6 * usual, v


def test_ruled_out_tokens(cuda_device):
    x, t = rows(6, 2000, 3)
    x[0, 100:1900] = -math.inf
    x[1] = -math.inf
    x[1, 1234] = 2.0                                     # one token left
    x[2] = -math.inf
    x[2, [5, 77]] = torch.tensor([1.0, 1.0])
    x[3] = -math.inf                                     # none left: no distribution
    x[4, ::2] = -math.inf
    t[:5] = torch.tensor([150, 1234, 6, 7, 1], dtype=torch.int32)   # the given token ruled out, the only one, ...
    check(cuda_device, x, t, 8)
    check(cuda_device, x, None, 32)


def test_rows_that_are_no_distribution(cuda_device):
    x, t = rows(6, 900, 4)
    x[0, 3], x[1, 899], x[2] = math.nan, math.inf, math.nan
    x[3, :] = -math.inf
    x[3, 500] = math.nan
    x[4] = math.inf
    check(cuda_device, x, t, 4)


def test_large_and_small_values(cuda_device):
    x, t = rows(5, 3000, 6)
    x[0] *= 1e30
    x[1] += 1e6
    x[2] *= 1e-30                                        # nearly uniform
    x[3] = -3e38
    x[3, 17] = 3e38
    x[4] = 1e-45 * torch.randint(0, 5, (3000,))          # (subnormal values are told apart)
    check(cuda_device, x, t, 16)


@pytest.mark.parametrize("rows_", [6, 800])
@pytest.mark.parametrize("offset", [9.5e6, 1.2e7, -3e7, 6e8])
def test_far_offsets(offset, rows_, cuda_device):
    # logits far from 0, whose steps in fp32 are 1 to 64: differences between them are exact
    g = torch.Generator().manual_seed(3)
    step = max(1.0, 2.0 ** (math.floor(math.log2(abs(offset))) - 23))
    x = (offset + step * torch.randint(-8, 9, (rows_, 700), generator=g)).float()
    check(cuda_device, x, torch.randint(0, 700, (rows_,), generator=g, dtype=torch.int32), 8)


def test_rows_not_asked_for_are_not_read(cuda_device):
    # as verification leaves them: [N, T] tokens with -1 behind those that stand; the rows there hold anything
    x, t = rows(12, 1500, 7)
    x, t = x.view(4, 3, 1500), t.view(4, 3)
    t[0, 1:], t[2, 2:], t[3, 0] = -1, -5, 1500
    y = x.clone()
    y[0, 1:], y[2, 2:], y[3, 0] = math.nan, math.inf, math.nan
    check(cuda_device, x, t, 5, gpu_logits=y.to(cuda_device), err=32)
    t[3, 0] = 2 ** 31 - 1
    check(cuda_device, x, t, 0, gpu_logits=y.to(cuda_device), err=32)


def test_strided_leading_dimensions(cuda_device):
    x, t = rows(12, 500, 8)
    wide = torch.zeros(12, 700, device=cuda_device)
    wide[:, :500] = x.to(cuda_device)
    check(cuda_device, x.view(4, 3, 500), t.view(4, 3), 3, gpu_logits=wide.view(4, 3, 700)[..., :500])
    # the last rows of a longer batch, and a batch of one
    check(cuda_device, x[9:], t[9:], 3, gpu_logits=wide[9:, :500])
    check(cuda_device, x[:1].view(1, 1, 500), t[:1].view(1, 1), 3, gpu_logits=wide[:1].view(1, 1, 700)[..., :500])


def test_graph_stream_and_repeated_calls(cuda_device):
    dev = cuda_device
    x, t = rows(40, 30000, 9)
    y, u = rows(40, 30000, 10)
    gx, gt = x.to(dev), t.to(dev)
    call = KdaLogprobsCall(gx, gt, num_top=6)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    call(side)
    side.synchronize()
    first = [v.clone() for v in (call.logprobs, call.ranks, call.entropy, call.top_ids, call.top_logprobs)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    gx.copy_(y), gt.copy_(u)
    g.replay()
    want = R.logprobs(y, u, 6)
    assert torch.equal(call.ranks.cpu(), want[1]) and torch.equal(call.top_ids.cpu(), want[3])
    gx.copy_(x), gt.copy_(t)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize(dev)
        for a, b in zip(first, (call.logprobs, call.ranks, call.entropy, call.top_ids, call.top_logprobs)):
            assert torch.equal(a, b)                     # the same bits every time


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_the_same_bits_under_load(dt, cuda_device):
    # more rows than CTAs, long enough for every stage of the ring to be used again: a copy that overtakes a reader shows
    # as a count that is off by a few
    g = torch.Generator(device=cuda_device).manual_seed(2)
    x = (torch.randn(1300, 60001, generator=g, device=cuda_device) * 3).to(dt)
    t = torch.randint(0, 60001, (1300,), generator=g, device=cuda_device, dtype=torch.int32)
    call = KdaLogprobsCall(x, t, num_top=20)
    call()
    results = lambda: (call.ranks, call.top_ids, call.logprobs, call.entropy, call.top_logprobs)  # noqa: E731
    first = [v.clone() for v in results()]
    xt = x.gather(1, t.long()[:, None])
    ranks = (x > xt).sum(1) + ((x == xt) & (torch.arange(60001, device=cuda_device) < t[:, None])).sum(1)
    assert torch.equal(first[0], ranks.int())
    for _ in range(20):
        call()
        for a, b in zip(first, results()):
            assert torch.equal(a, b)


def test_far_rows(cuda_device):
    # offsets past 2^31 elements
    V, R_ = 200000, 11000
    x, t = rows(3, V, 12, torch.bfloat16)
    big = torch.empty(R_, V, dtype=torch.bfloat16, device=cuda_device)
    tok = torch.full((R_,), -1, dtype=torch.int32, device=cuda_device)
    at = [0, 10900, 10999]
    big[at], tok[at] = x.to(cuda_device), t.to(cuda_device)
    got = kda_logprobs(big, tok, num_top=4)
    want = R.logprobs(x, t, 4)
    assert torch.equal(got[1][at].cpu(), want[1]) and torch.equal(got[3][at].cpu(), want[3])
    same(got[0][at], want[0], INNER + want[0].abs() * 2.0 ** -22)
    rest = torch.ones(R_, dtype=torch.bool)
    rest[at] = False
    assert (got[0].cpu()[rest] == 0).all() and (got[3].cpu()[rest] == -1).all() and (got[1].cpu()[rest] == -1).all()


def test_no_rows_and_refusals(cuda_device):
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=cuda_device)  # noqa: E731
    assert kda_logprobs(z(0, 9), z(0, dt=torch.int32), num_top=2)[3].shape == (0, 2)
    t = z(4, dt=torch.int32)
    for bad in (lambda: kda_logprobs(z(4, 9, dt=torch.float16), t), lambda: kda_logprobs(z(4, 9), t.long()),
                lambda: kda_logprobs(z(4, 9), t[:3]), lambda: kda_logprobs(z(4, 9), t, num_top=33),
                lambda: kda_logprobs(z(4, 9), t, num_top=-1), lambda: kda_logprobs(z(9), t[:1]),
                lambda: kda_logprobs(z(4, 0), t), lambda: kda_logprobs(z(9, 4).t(), t),
                lambda: kda_logprobs(z(2, 3, 9)[:, :2], z(2, 2, dt=torch.int32)), lambda: kda_logprobs(z(4, 9).cpu(), t),
                lambda: kda_logprobs(z(1, 9).expand(4, 9), t)):
        with pytest.raises((TypeError, ValueError)):
            bad()
