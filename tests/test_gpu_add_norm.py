"""Residual addition with norm and 8-bit output against 64 bits."""
import pytest
import torch

import layer_reference as R
from linear_attention_decode_04_gb300 import KdaAddNormCall, kda_add_norm

pytestmark = pytest.mark.gpu

# fp32 inside: a sum of squares adds at most 64 terms a thread and two trees of five, half of which a root keeps; six
# more roundings: below 2^-18 of the value
INNER = 2.0 ** -18


def inputs(T, D, seed, residual=True, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, D, generator=g) * scale).bfloat16()
    r = (torch.randn(T, D, generator=g) * torch.exp(torch.randn(D, generator=g)) * scale).bfloat16() if residual else None
    return x, r, torch.rand(D, generator=g) + 0.5


def wide(t, pad, fill):
    """The rows of t inside wider ones: (view, whole)"""
    w = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=torch.float32, device=t.device).to(t.dtype)
    w[:, :t.shape[1]] = t
    return w[:, :t.shape[1]], w


def outputs(T, D, dev, pad=0, scale_pad=0):
    new = lambda dt: wide(torch.zeros(T, D, device=dev).to(dt), pad, 3.0)[0]  # noqa: E731
    return dict(residual_out=new(torch.bfloat16), out=new(torch.bfloat16), out_q=new(torch.float8_e4m3fn),
                out_scale=torch.full((T,), 5.0, device=dev))


def check(got, x, weight=None, residual=None, eps=1e-6, norm=True):
    h, y, s = R.add_norm(x, weight, residual, eps, norm)
    tol = y.abs() * (R.BF16 + INNER) + 1e-38
    assert ((got["out"].cpu().double() - y).abs() <= tol).all()
    assert ((got["residual_out"].cpu().double() - h).abs() <= h.abs() * (R.BF16 + R.FP32) + 1e-38).all()
    sc = got["out_scale"].cpu().double()
    assert ((sc - s).abs() <= s * INNER).all()
    v, code = y / s[:, None], got["out_q"].cpu().double()
    assert ((code - v).abs() <= v.abs() * (R.E4M3 + INNER) + R.E4M3_TINY).all()
    assert (code.abs().amax(-1)[s > 2 * R.SCALE_FLOOR / 448] == 448).all()


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("T, D", [(1, 8), (3, 16), (2, 248), (5, 256), (4, 264), (7, 2048), (300, 2056), (33, 4608),
                                  (9, 6144), (5, 6152), (700, 1000), (3, 8192), (2, 8200), (3, 16384), (2, 32760),
                                  (2, 32768)])
def test_matches_64_bits(T, D, residual, cuda_device):
    x, r, w = inputs(T, D, T + D, residual)
    got = outputs(T, D, cuda_device)
    kda_add_norm(x.to(cuda_device), weight=w.to(cuda_device), residual=None if r is None else r.to(cuda_device), **got)
    check(got, x, w, r)


@pytest.mark.parametrize("T, D", [(1, 1536), (2, 1544), (3, 504), (5, 1024), (4097, 512), (2049, 1288), (6, 520)])
def test_short_rows(T, D, cuda_device):
    # rows of a warp each, several to a CTA, and the first that are not
    x, r, w = inputs(T, D, T * D)
    got = outputs(T, D, cuda_device, pad=8)
    kda_add_norm(x.to(cuda_device), weight=w.to(cuda_device), residual=r.to(cuda_device), **got)
    check(got, x, w, r)


@pytest.mark.parametrize("T, D", [(1, 8), (3, 264), (5, 6144), (41, 4608), (2, 32768)])
def test_without_norm_or_weight(T, D, cuda_device):
    x, r, _ = inputs(T, D, T * D)
    got = outputs(T, D, cuda_device)
    kda_add_norm(x.to(cuda_device), residual=r.to(cuda_device), norm=False, **got)
    check(got, x, None, r, norm=False)
    kda_add_norm(x.to(cuda_device), eps=1e-3, **got)
    check(got, x, eps=1e-3)


@pytest.mark.parametrize("which", ["out", "residual_out", "q", "out+q", "out+residual_out"])
def test_any_set_of_results(which, cuda_device):
    # what is left out changes nothing in what is asked for
    x, r, w = inputs(5, 2056, 3)
    g = dict(weight=w.to(cuda_device), residual=r.to(cuda_device))
    every, some = outputs(5, 2056, cuda_device), outputs(5, 2056, cuda_device)
    kda_add_norm(x.to(cuda_device), **g, **every)
    names = [n for part in which.split("+") for n in (("out_q", "out_scale") if part == "q" else (part,))]
    kda_add_norm(x.to(cuda_device), **g, **{n: some[n] for n in names})
    for n in names:
        assert torch.equal(some[n].view(torch.uint8), every[n].view(torch.uint8))


def test_strided_rows_leave_the_rest(cuda_device):
    T, D = 37, 1032
    x, r, w = inputs(T, D, 11)
    dev = cuda_device
    got = outputs(T, D, dev, pad=24)
    kda_add_norm(wide(x.to(dev), 8, 9.0)[0], weight=w.to(dev), residual=wide(r.to(dev), 40, 9.0)[0], **got)
    check(got, x, w, r)
    for n in ("out", "residual_out", "out_q"):
        whole = torch.as_strided(got[n], (T, D + 24), (D + 24, 1))
        assert (whole[:, D:].float() == 3.0).all(), n


@pytest.mark.parametrize("T", [1, 5, 2000])
def test_in_place(T, cuda_device):
    # residual_out over residual and out over x: the stream and the layer's input in the same two buffers
    D, dev = 2048, cuda_device
    x, r, w = inputs(T, D, T)
    for swap in (False, True):
        gx, gr = x.to(dev), r.to(dev)
        got = outputs(T, D, dev)
        got["residual_out"], got["out"] = (gx, gr) if swap else (gr, gx)
        kda_add_norm(gx, weight=w.to(dev), residual=gr, **got)
        check(got, x, w, r)


def test_rows_that_are_not_finite_or_empty(cuda_device):
    D, dev = 520, cuda_device
    x, r, w = inputs(8, D, 5)
    x[0, 7], x[1, 500], r[2, 0] = float("nan"), float("inf"), float("-inf")
    x[3], r[3] = 0, 0                                   # nothing in the row
    x[4], r[4] = 1e-38, 0                               # squares and codes far below the rest
    x[5], r[5] = 3e38, 3e38                             # the sum passes fp32's range
    for norm in (True, False):
        got = outputs(8, D, dev)
        kda_add_norm(x.to(dev), weight=w.to(dev) if norm else None, residual=r.to(dev), norm=norm, **got)
        h, y, s = R.add_norm(x, w if norm else None, r, norm=norm)
        sc = got["out_scale"].cpu().double()
        assert sc[[0, 1, 2]].isnan().all()
        code = got["out_q"].cpu().double()
        assert (code[3] == 0).all() and abs(sc[3] * 448 * 2.0 ** 100 - 1) <= R.FP32   # (rounded to fp32)
        rows = [3, 4, 6, 7]
        assert ((sc[rows] - s[rows]).abs() <= s[rows] * INNER).all()
        v = (y / s[:, None])[rows]
        assert ((code[rows] - v).abs() <= v.abs() * (R.E4M3 + INNER) + R.E4M3_TINY).all()
        d = (got["out"].cpu().double() - y)[rows].abs()
        assert (d <= y[rows].abs() * (R.BF16 + INNER) + 1e-38).all()
        assert sc[5].isnan() or norm                    # (an infinite sum of squares makes the row zeros)


@pytest.mark.parametrize("T, D, scale", [(4096, 512, 1.0), (2000, 6144, 1e-30), (700, 32768, 1e34), (3000, 520, 3e-5)])
def test_codes_are_quotients_by_the_stored_scale(T, D, scale, cuda_device):
    # without the norm y is a sum that fp32 holds, and the codes have one value each: the fp32 quotient, rounded to e4m3
    x, r, _ = inputs(T, D, T + D, scale=scale)
    got = outputs(T, D, cuda_device)
    del got["out"]
    kda_add_norm(x.to(cuda_device), residual=r.to(cuda_device), norm=False, **got)
    y = x.float() + r.float()
    want = y.abs().amax(-1) * (torch.tensor(1.0) / 448)
    assert torch.equal(got["out_scale"].cpu(), want)
    codes = (y / want[:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(got["out_q"].cpu().view(torch.uint8), codes.view(torch.uint8))
    # what a product with the rounded reciprocal would get wrong is among them
    assert (codes.view(torch.uint8) != (y * (448 / y.abs().amax(-1))[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)).any()


@pytest.mark.parametrize("eps", [1e-6, 0.0, 1e-40])
@pytest.mark.parametrize("T, D", [(9, 264), (9, 512), (9, 520), (9, 6152), (9, 32768)])
def test_squares_past_the_range_of_fp32(T, D, eps, cuda_device):
    x, r, w = inputs(T, D, D)
    # rows as a whole, and one channel of the next ones: squares past 2^128, and far below 2^-126
    for i, size in enumerate((1e20, 1e37, 1e-22, 1e-36)):
        x[2 * i], r[2 * i] = (x[2 * i].float() * size).bfloat16(), (r[2 * i].float() * size).bfloat16()
        x[2 * i + 1, 5] = size
    got = outputs(T, D, cuda_device)
    kda_add_norm(x.to(cuda_device), weight=w.to(cuda_device), residual=r.to(cuda_device), eps=eps, **got)
    finite = torch.isfinite(x.float() + r.float()).all(-1)     # (some channels of the rows of 1e37 are not, in bf16 already)
    assert got["out_scale"].cpu()[~finite].isnan().all() and finite.sum() >= 7
    check({k: v.float()[finite.to(v.device)] for k, v in got.items()}, x[finite], w, r[finite], torch.tensor(eps).item())
    assert (got["out_scale"].cpu()[finite] > 0).all()


def test_rows_of_zeros_and_infinities(cuda_device):
    # 0 / 0 without eps; an infinite sum leaves finite channels 0 and is NaN itself
    x = torch.zeros(3, 520).bfloat16()
    x[1, 3], x[2] = 3e38, 1e-20
    r = torch.zeros_like(x)
    r[1, 3] = 3e38
    for eps in (0.0, 1e-6):
        got = outputs(3, 520, cuda_device)
        kda_add_norm(x.to(cuda_device), residual=r.to(cuda_device), eps=eps, **got)
        out = got["out"].cpu().float()
        assert out[0].isnan().all() if eps == 0 else (out[0] == 0).all()
        assert out[1, 3].isnan() and (out[1, :3] == 0).all() and (out[1, 4:] == 0).all()
        assert got["out_scale"][1].isnan()
        want = 1.0 if eps == 0 else 1e-17
        assert ((out[2].double() - want).abs() <= want * 2.0 ** -7).all()


def test_graph_stream_and_repeated_rows(cuda_device):
    # a row's results do not depend on the rows beside it, the stream or a replay
    dev = cuda_device
    x, r, w = inputs(64, 4608, 21)
    gx, gr, gw = x.to(dev), r.to(dev), w.to(dev)
    one = outputs(64, 4608, dev)
    KdaAddNormCall(gx, weight=gw, residual=gr, **one)()
    many = outputs(4096, 4608, dev)
    rep = lambda t: t.repeat(64, 1)  # noqa: E731
    call = KdaAddNormCall(rep(gx), weight=gw, residual=rep(gr), **many)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    call(side)
    side.synchronize()
    for n in one:
        a = one[n].view(torch.uint8).view(64, -1)
        assert torch.equal(many[n].view(torch.uint8).view(64, 64, -1), a.expand(64, 64, -1)), n
    for t in many.values():
        t.view(torch.uint8).zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    g.replay()
    torch.cuda.synchronize(dev)
    for n in one:
        a = one[n].view(torch.uint8).view(64, -1)
        assert torch.equal(many[n].view(torch.uint8).view(64, 64, -1), a.expand(64, 64, -1)), n


def test_no_rows(cuda_device):
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=cuda_device)  # noqa: E731
    kda_add_norm(e(0, 64), out=e(0, 64))


def test_refusals(cuda_device):
    e = lambda *s, dt=torch.bfloat16: torch.zeros(*s, device=cuda_device).to(dt)  # noqa: E731
    x, f8 = e(4, 64), torch.float8_e4m3fn
    kda_add_norm(x, out=e(4, 64))
    for kw in (dict(), dict(out=e(4, 64, dt=torch.float16)), dict(out=e(3, 64)), dict(out=e(4, 72)),
               dict(out_q=e(4, 64, dt=f8)), dict(out_q=e(4, 64), out_scale=e(4, dt=torch.float32)),
               dict(out=e(4, 64), weight=e(64)), dict(out=e(4, 64), weight=e(64, dt=torch.float32), norm=False),
               dict(out=e(64, 4).t()), dict(out=x.view(-1)[:0].view(0, 64)), dict(out=e(4, 64).cpu())):
        with pytest.raises((TypeError, ValueError)):
            kda_add_norm(x, **kw)
    with pytest.raises(ValueError, match="multiple of 8"):
        kda_add_norm(e(4, 60), out=e(4, 60))
    buf = e(5, 64)
    with pytest.raises(ValueError, match="overlaps"):
        kda_add_norm(buf[:4], out=buf[1:])
    y = e(4, 64)
    with pytest.raises(ValueError, match="overlaps"):
        kda_add_norm(x, out=y, residual_out=y)
    both = e(4, 128)
    kda_add_norm(both[:, :64], out=both[:, 64:])        # columns of the same rows that do not meet
    with pytest.raises(ValueError, match="overlaps"):
        kda_add_norm(both[:, :64], out=both[:, 8:72])
