"""Matrix products with epilogues against 64 bits."""
import math

import pytest
import torch

import layer_reference as R
from linear_attention_decode_04_gb300 import KdaLinearCall, kda_linear

pytestmark = pytest.mark.gpu

ACTS = [None, "silu", "gelu", "silu_gated"]
F8 = torch.float8_e4m3fn


def whole_numbers(shape, g, e4m3):
    # products of these are exact in any order and sum
    return torch.randint(-3, 4, shape, generator=g).float().to(F8 if e4m3 else torch.bfloat16)


def padded(t, pad, dev, fill=0.0):
    """t on the device, as columns of wider rows"""
    w = torch.full((t.shape[0], t.shape[1] + pad), fill).to(t.dtype).to(dev)
    w[:, :t.shape[1]] = t.to(dev)
    return w[:, :t.shape[1]]


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("M, N, K", [(1, 1, 16), (1, 128, 128), (3, 130, 144), (16, 256, 4096), (17, 129, 272), (33, 64, 64),
                                     (64, 1000, 2048), (65, 300, 1008), (128, 128, 8192), (129, 640, 400), (256, 384, 640),
                                     (257, 2000, 160), (700, 259, 336), (1100, 5000, 96)])
def test_whole_numbers_are_exact(M, N, K, e4m3, cuda_device):
    # every row tile, clusters of one to eight CTAs, ragged ends of each dimension
    g = torch.Generator().manual_seed(M + N + K)
    x, w = whole_numbers((M, K), g, e4m3), whole_numbers((N, K), g, e4m3)
    sx = sw = None
    if e4m3:
        sx, sw = (2.0 ** torch.randint(-3, 4, (n,), generator=g).float() for n in (M, N))
    out = torch.full((M, N), float("nan"), device=cuda_device)
    d = lambda t: None if t is None else t.to(cuda_device)  # noqa: E731
    kda_linear(d(x), d(w), out, x_scale=d(sx), weight_scale=d(sw))
    want = x.float() @ w.float().t()
    if e4m3:
        want = want * sx[:, None] * sw
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("e4m3, M, N, K", [
    (False, 17, 16, 16), (False, 2, 17, 592), (False, 22, 16, 592), (False, 2, 19, 1168), (False, 20, 29, 1168),   # 16 rows
    (False, 27, 9742, 16), (True, 617, 386, 16), (False, 27, 4897, 1456), (False, 311, 401, 1264), (False, 19, 2472, 4096),
    (False, 762, 16, 3536),                                                                                        # 32 rows
    (False, 52, 9788, 32), (True, 816, 667, 16), (False, 50, 5323, 2624), (False, 2484, 18, 2576), (False, 51, 2532, 6032),
    (False, 1364, 20, 6048),                                                                                       # 64 rows
    (False, 102, 9779, 16), (False, 986, 1158, 16), (False, 4911, 21, 3472),                                       # 128 rows
    (False, 108, 9959, 416), (False, 1225, 973, 368), (False, 117, 4895, 2496), (False, 2842, 130, 2128),
    (False, 99, 2463, 5680), (False, 1217, 154, 5824),                                                             # pairs, 128 rows
    (False, 203, 9760, 16), (False, 1310, 1676, 16), (True, 300, 20000, 256), (True, 2900, 1537, 384)])            # 256 rows
def test_every_tile_and_share_of_k(e4m3, M, N, K, cuda_device):
    # one row tile and several, a tile's products in one, two and four parts; results in fp32, and in bf16 onto a residual
    # in rows on no boundary: sums are whole numbers below 2^24, so there is one right answer
    g = torch.Generator().manual_seed(M + N + K)
    x, w = whole_numbers((M, K), g, e4m3), whole_numbers((N, K), g, e4m3)
    one = dict(x_scale=torch.ones(M, device=cuda_device), weight_scale=torch.ones(N, device=cuda_device)) if e4m3 else {}
    want = x.float() @ w.float().t()
    xd, wd = x.to(cuda_device), w.to(cuda_device)
    for early in (False, True):
        out = torch.full((M, N), float("nan"), device=cuda_device)
        kda_linear(xd, wd, out, early_weight=early, **one)
        assert torch.equal(out.cpu(), want)
    res = torch.randint(-100, 101, (M, N), generator=g).bfloat16()
    want = (want + res.float()).bfloat16()
    for at in (0, 1, 2, 3):
        for pitch in (N + 5, (N + 15) // 8 * 8):
            buf = torch.full((M, pitch), 3.0, dtype=torch.bfloat16, device=cuda_device)
            view = buf[:, at:at + N]
            view.copy_(res.to(cuda_device))
            kda_linear(xd, wd, view, residual=view, **one)
            assert torch.equal(view.cpu(), want), (at, pitch)
            assert (buf[:, :at] == 3.0).all() and (buf[:, at + N:] == 3.0).all(), (at, pitch)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("e4m3, M, N, K", [(True, 18, 16, 16), (False, 17, 26, 464), (False, 36, 30, 912), (False, 614, 800, 16),
                                           (False, 1282, 22, 976), (False, 632, 26, 2480), (True, 1246, 824, 16),
                                           (False, 2682, 26, 1904), (False, 1451, 22, 4768), (False, 1686, 1290, 16),
                                           (True, 1327, 3590, 16), (True, 300, 6002, 272)])
def test_every_gated_tile(e4m3, M, N, K, f32, cuda_device):
    p = problem(M, N, K, e4m3, "silu_gated", True, not f32, M)
    d = {k: v.to(cuda_device) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    for pad in (0, 3):
        out = torch.full((M, N // 2 + pad), 9.0, dtype=torch.float32 if f32 else torch.bfloat16, device=cuda_device)
        kda_linear(out=out[:, :N // 2], **d)
        close(out[:, :N // 2], p, not f32)
        assert (out[:, N // 2:] == 9.0).all()


@pytest.mark.parametrize("e4m3, M, N, K", [(False, 2455, 19, 11456), (True, 2455, 2, 22912)])
def test_tiles_of_128_rows_in_four_parts(e4m3, M, N, K, cuda_device):
    test_every_tile_and_share_of_k(e4m3, M, N, K, cuda_device)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("e4m3, M, N, K", [(True, 1300, 3600, 1600), (False, 1300, 3600, 800), (False, 700, 9008, 776)])
def test_gated_tiles_of_two_warpgroups(e4m3, M, N, K, f32, cuda_device):
    test_every_gated_tile(e4m3, M, N, K, f32, cuda_device)


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("K", [1, 7, 31, 33, 65, 127, 130, 1001])
@pytest.mark.parametrize("M, N", [(3, 5), (40, 200), (300, 260)])
def test_any_k(M, N, K, e4m3, cuda_device):
    # rows that end inside 16 bytes, with something else behind them
    g = torch.Generator().manual_seed(K)
    x, w = whole_numbers((M, K), g, e4m3), whole_numbers((N, K), g, e4m3)
    one = dict(x_scale=torch.ones(M, device=cuda_device), weight_scale=torch.ones(N, device=cuda_device)) if e4m3 else {}
    pad = -K % 16 + 16
    out = torch.full((M, N), float("nan"), device=cuda_device)
    kda_linear(padded(x, pad, cuda_device, 2.0), padded(w, pad, cuda_device, math.nan), out, **one)
    assert torch.equal(out.cpu(), x.float() @ w.float().t())


@pytest.mark.parametrize("f32, e4m3, M, N, K", [
    (True, False, 4, 700, 9008), (True, False, 3, 130, 40008), (True, False, 30, 9800, 2112), (True, False, 200, 2570, 4400),
    (True, False, 1400, 300, 2500 // 8 * 8), (True, False, 700, 9000, 2056), (True, False, 1300, 5130, 4104),
    (True, True, 9, 1000, 20000), (True, True, 600, 520, 33008), (False, False, 2, 20, 280000), (False, False, 500, 150, 66000)])
def test_long_sums_in_parts(f32, e4m3, M, N, K, cuda_device):
    # more of k than is summed up at a time; tiles in turn, tiles shared by CTAs
    g = torch.Generator().manual_seed(K)
    x, w = whole_numbers((M, K), g, e4m3), whole_numbers((N, K), g, e4m3)
    one = dict(x_scale=torch.ones(M, device=cuda_device), weight_scale=torch.ones(N, device=cuda_device)) if e4m3 else {}
    want = x.float() @ w.float().t()
    assert want.abs().max() < 2 ** 24
    out = torch.full((M, N), float("nan"), dtype=torch.float32 if f32 else torch.bfloat16, device=cuda_device)
    kda_linear(x.to(cuda_device), w.to(cuda_device), out, **one)
    assert torch.equal(out.cpu(), want.to(out.dtype))


@pytest.mark.parametrize("M, N, K", [(5, 200, 4112), (40, 130, 9000), (130, 4000, 2200), (300, 600, 4104), (600, 9000, 2112)])
def test_long_gated_sums_in_parts(M, N, K, cuda_device):
    p = problem(M, N, K, False, "silu_gated", True, False, K)
    out = torch.full((M, N // 2), float("nan"), device=cuda_device)
    kda_linear(out=out, **{k: v.to(cuda_device) if isinstance(v, torch.Tensor) else v for k, v in p.items()})
    close(out, p, False)


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("M, N", [(16, 256), (150, 512), (256, 2048)])
def test_long_sums_are_not_shortened(M, N, e4m3, cuda_device):
    # The tensor cores cut sums towards zero: half a step each of 2^-23 of the sum so far, whose magnitude grows with the
    # root of the number of products.  Over 56 additions (896 of k) that takes 2/3 * 56 * 2^-24 * 0.72 = 1.6e-6 of a sum,
    # which is what any k may be off by in parts of 896; 16,384 in one go would be 18 times that.
    K = 16384
    p = problem(M, N, K, e4m3, None, False, False, 11)
    d = {k: v.to(cuda_device) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    out = torch.zeros(M, N, device=cuda_device)
    kda_linear(out=out, **d)
    y = d["x"].double() @ d["weight"].double().t()
    if e4m3:
        y = y * d["x_scale"].double()[:, None] * d["weight_scale"].double()
    assert ((out.double() - y).norm() / y.norm()).item() < 2.0 ** -19


def problem(M, N, K, e4m3, act, bias, residual, seed):
    g = torch.Generator().manual_seed(seed)
    p = dict(x=torch.randn(M, K, generator=g), weight=torch.randn(N, K, generator=g) / math.sqrt(K))
    if e4m3:
        p["x_scale"], p["weight_scale"] = (p[n].abs().amax(-1) / 448 for n in ("x", "weight"))
        p["x"], p["weight"] = ((p[n] / p[s][:, None]).to(F8) for n, s in (("x", "x_scale"), ("weight", "weight_scale")))
    else:
        p["x"], p["weight"] = p["x"].bfloat16(), p["weight"].bfloat16()
    if bias:
        p["bias"] = torch.randn(N, generator=g)
    if residual:
        p["residual"] = torch.randn(M, N // 2 if act == "silu_gated" else N, generator=g).bfloat16()
    p["activation"] = act
    return p


def close(got, p, bf16):
    want, tol = R.linear(**p)
    d = (got.cpu().double() - want).abs()
    bad = d > tol + (want.abs() + tol) * (R.BF16 if bf16 else 0) + 1e-37
    assert not bad.any(), (d[bad][:5], want[bad][:5], bad.nonzero()[:5])


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M, N, K", [(5, 200, 528), (40, 1026, 256), (100, 386, 1024), (300, 514, 304)])
def test_epilogues(M, N, K, act, e4m3, f32, cuda_device):
    for bias, residual in ((True, True), (False, True), (True, False)):
        p = problem(M, N, K, e4m3, act, bias, residual, M + N)
        width = N // 2 if act == "silu_gated" else N
        out = torch.full((M, width), float("nan"), dtype=torch.float32 if f32 else torch.bfloat16, device=cuda_device)
        kda_linear(out=out, **{k: v.to(cuda_device) if isinstance(v, torch.Tensor) else v for k, v in p.items()})
        close(out, p, not f32)


@pytest.mark.parametrize("e4m3", [True, False])
def test_strides_and_in_place_residual(e4m3, cuda_device):
    M, N, K, dev = 70, 331, 208, cuda_device
    p = problem(M, N, K, e4m3, None, True, True, 9)
    q = {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    q["x"], q["weight"] = padded(p["x"], 48, dev, 2.0), padded(p["weight"], 16, dev, 2.0)
    buf = torch.full((M, N + 5), 7.0, dtype=torch.bfloat16, device=dev)
    buf[:, :N] = p["residual"].to(dev)
    q["residual"] = buf[:, :N]
    kda_linear(out=buf[:, :N], **q)                     # onto the residual itself, rows on no boundary
    close(buf[:, :N], p, True)
    assert (buf[:, N:] == 7.0).all()


@pytest.mark.parametrize("M, N", [(1, 7), (20, 130), (300, 1000)])
def test_nothing_but_its_rows_is_written(M, N, cuda_device):
    g = torch.Generator().manual_seed(1)
    x, w = whole_numbers((M, 64), g, False), whole_numbers((N, 64), g, False)
    whole = torch.full((M + 2, N + 3), 5.0, device=cuda_device)
    kda_linear(x.to(cuda_device), w.to(cuda_device), whole[1:M + 1, 1:N + 1])
    assert torch.equal(whole[1:M + 1, 1:N + 1].cpu(), x.float() @ w.float().t())
    whole[1:M + 1, 1:N + 1] = 5.0
    assert (whole == 5.0).all()


@pytest.mark.parametrize("M", [3, 40, 400])
def test_rows_that_are_not_finite_stay_alone(M, cuda_device):
    N, K = 300, 512
    p = problem(M, N, K, True, "silu", False, False, 3)
    p["x_scale"][1] = math.nan
    p["x"][2, 5] = math.nan
    out = torch.zeros(M, N, device=cuda_device)
    kda_linear(out=out, **{k: v.to(cuda_device) if isinstance(v, torch.Tensor) else v for k, v in p.items()})
    assert out[1:3].isnan().all()
    rest = [i for i in range(M) if i not in (1, 2)]
    q = {**p, "x": p["x"].view(torch.uint8)[rest].view(F8), "x_scale": p["x_scale"][rest]}
    close(out[rest], q, False)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M, N", [(5, 64), (40, 300), (300, 520)])
def test_values_that_are_not_finite(M, N, act, f32, cuda_device):
    # NaN stays NaN through every activation; infinity is its own gelu and silu, and gelu's lower tail ends at 0
    x, w = torch.zeros(M, 64, dtype=torch.bfloat16), torch.ones(N, 64, dtype=torch.bfloat16)
    x[:, 0] = 1.0
    x[0, 3], x[1, 3], x[2, 3], x[3, 3] = math.nan, math.inf, -math.inf, -300.0
    width = N // 2 if act == "silu_gated" else N
    out = torch.full((M, width), 5.0, dtype=torch.float32 if f32 else torch.bfloat16, device=cuda_device)
    kda_linear(x.to(cuda_device), w.to(cuda_device), out, activation=act)
    got = out.cpu().double()
    assert got[0].isnan().all()
    assert (got[1] == math.inf).all()
    assert act not in (None, "gelu") or (got[2] == (-math.inf if act is None else 0)).all()
    assert act is None or (got[3].abs() < 1e-37).all()
    one = {None: 1.0, "silu": 1 / (1 + math.exp(-1)), "gelu": 0.5 * (1 + math.erf(math.sqrt(0.5))), "silu_gated": 1 / (1 + math.exp(-1))}[act]
    assert ((got[4:] - one).abs() <= (2.0 ** -18 if f32 else 2.0 ** -8)).all()


def test_rows_do_not_depend_on_one_another_in_a_tile_size(cuda_device):
    # the same row gives the same bits wherever it stands in a batch that takes the same variant
    dev = cuda_device
    p = problem(60, 500, 1024, True, None, False, False, 4)
    d = {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    a, b = torch.zeros(60, 500, device=dev), torch.zeros(60, 500, device=dev)
    kda_linear(out=a, **d)
    perm = torch.randperm(60)
    kda_linear(out=b, **{**d, "x": d["x"].view(torch.uint8)[perm].view(F8), "x_scale": d["x_scale"][perm]})
    assert torch.equal(a[perm], b)


def test_graph_stream_and_early_weight(cuda_device):
    dev = cuda_device
    p = problem(8, 4608, 2048, True, None, False, False, 6)
    d = {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    want = torch.zeros(8, 4608, device=dev)
    kda_linear(out=want, **d)
    for early in (False, True):
        out = torch.zeros(8, 4608, device=dev)
        call = KdaLinearCall(out=out, early_weight=early, **d)
        side = torch.cuda.Stream(dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        call(side)
        side.synchronize()
        assert torch.equal(out, want)
        x2 = torch.zeros_like(out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(5):
                call()
            x2.copy_(out)
        out.zero_()
        g.replay()
        torch.cuda.synchronize(dev)
        assert torch.equal(x2, want) and torch.equal(out, want)


def test_chain_of_products(cuda_device):
    # each call reads what the one ahead of it wrote, with weights asked for early
    dev = cuda_device
    g = torch.Generator().manual_seed(8)
    w = [whole_numbers((128, 128), g, False) for _ in range(4)]
    x = whole_numbers((20, 128), g, False)
    bufs = [x.to(dev)] + [torch.zeros(20, 128, dtype=torch.bfloat16, device=dev) for _ in w]
    wd = [t.to(dev) for t in w]
    for rep in range(20):
        for i, t in enumerate(wd):
            kda_linear(bufs[i], t, bufs[i + 1], early_weight=True)
        want = x
        for t in w:
            want = (want.float() @ t.float().t()).bfloat16()
        # (sums pass 2^24 from the third product on: products of rounded values, one order of sums per variant)
        got = [b.cpu().double() for b in bufs]
        for i, t in enumerate(w):
            y, tol = R.linear(got[i], t)
            assert ((got[i + 1] - y).abs() <= tol + (y.abs() + tol) * R.BF16).all(), (rep, i)


def test_no_rows(cuda_device):
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=cuda_device)  # noqa: E731
    kda_linear(e(0, 64), e(32, 64), e(0, 32))


def test_refusals(cuda_device):
    e = lambda *s, dt=torch.bfloat16: torch.zeros(*s, device=cuda_device).to(dt)  # noqa: E731
    f32 = lambda *s: e(*s, dt=torch.float32)  # noqa: E731
    x, w, out = e(4, 64), e(32, 64), e(4, 32)
    kda_linear(x, w, out)
    for kw in (dict(x=x.float()), dict(weight=w.to(F8)), dict(weight=e(32, 72)), dict(out=e(4, 33)), dict(out=e(3, 32)),
               dict(out=e(4, 32, dt=torch.float16)), dict(x_scale=f32(4)), dict(bias=e(32)), dict(bias=f32(31)),
               dict(residual=f32(4, 32)), dict(residual=e(4, 31)), dict(activation="tanh"), dict(out=out.cpu()),
               dict(x=x.to(F8), weight=w.to(F8)), dict(x=x.to(F8), weight=w.to(F8), x_scale=f32(4), weight_scale=f32(31)),
               dict(activation="silu_gated"), dict(activation="silu_gated", weight=e(33, 64), out=e(4, 16))):
        with pytest.raises((TypeError, ValueError)):
            kda_linear(**{**dict(x=x, weight=w, out=out), **kw})
    both = e(4, 96)
    with pytest.raises(ValueError, match="overlaps"):
        kda_linear(both[:, :64], w, both[:, 32:64])
    kda_linear(both[:, :64], w, both[:, 64:])
    from linear_attention_decode_04_gb300 import KdaError
    with pytest.raises(KdaError, match="aligned"):
        kda_linear(e(4, 65)[:, :64], w, out)
