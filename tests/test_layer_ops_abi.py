"""The operators of ``layer_ops`` on the host: struct mirrors, argument codes of
the C ABI (before any CUDA call, with pointers that are never dereferenced),
refusals of the Python calls, and the references that the GPU tests use."""
import ctypes
import math

import pytest
import torch

import layer_reference as R
from linear_attention_decode_04_gb300 import binding, kda_add_norm, kda_linear, kda_logprobs
from linear_attention_decode_04_gb300 import build as B
from linear_attention_decode_04_gb300 import layer_ops as L
from test_step_ops_abi import caller, header_fields

OK, NULLPTR, SHAPE, ALIGN, FLAGS = 0, -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    B.build()
    return binding.load_library()


@pytest.mark.parametrize("header, struct", [("kda_add_norm.h", L.KdaAddNormArgs), ("kda_linear.h", L.KdaLinearArgs),
                                            ("kda_logprobs.h", L.KdaLogprobsArgs)])
def test_struct_mirrors(header, struct):
    assert header_fields(header, struct.__name__) == [f for f, _ in struct._fields_]


def test_add_norm_codes(lib):
    names = ("x", "residual", "weight", "residual_out", "out", "out_q", "out_scale")
    at = {n: 0x100000 * (i + 1) for i, n in enumerate(names)}
    strides = {n + "_row_stride": 64 for n in ("x", "residual", "residual_out", "out", "out_q")}
    call = caller(lib, "kda_add_norm", L.KdaAddNormArgs, dict(T=4, D=64, eps=1e-6, **at, **strides))
    for kw in (dict(T=-1), dict(D=0), dict(D=60), dict(D=32776), dict(eps=-1.0), dict(eps=math.nan),
               dict(out=at["residual_out"]), dict(out_q=at["out"]), dict(out_q=at["x"]),
               dict(out=at["x"], out_row_stride=72), dict(residual_out=at["residual"], residual_out_row_stride=128),
               *[{s: 56} for s in strides]):
        assert call(**kw) == SHAPE, kw
    assert call(flags=2) == FLAGS and call(flags=1) == FLAGS          # unknown; a weight without the norm
    assert call(T=0) == OK
    for kw in (dict(x=None), dict(out_scale=None), dict(out_q=None),
               dict(residual_out=None, out=None, out_q=None, out_scale=None)):
        assert call(**kw) == NULLPTR, kw
    for kw in (dict(x=at["x"] + 8), dict(residual=at["residual"] + 2), dict(out=at["out"] + 8), dict(out_q=at["out_q"] + 4),
               dict(weight=at["weight"] + 4), dict(out_scale=at["out_scale"] + 2), dict(residual_out=at["residual_out"] + 8),
               *[{s: 68} for s in strides]):
        assert call(**kw) == ALIGN, kw


def test_linear_codes(lib):
    names = ("x", "weight", "x_scale", "weight_scale", "bias", "residual", "out", "err_flag")
    at = {n: 0x1000000 * (i + 1) for i, n in enumerate(names)}
    good = dict(M=4, N=64, K=32, flags=1, x_row_stride=32, weight_row_stride=32, residual_row_stride=64, out_row_stride=64)
    call = caller(lib, "kda_linear", L.KdaLinearArgs, dict(**good, **at))
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(N=2 ** 24 + 1), dict(K=2 ** 24 + 1), dict(activation=4), dict(activation=-1),
               dict(activation=3, N=63), dict(x_row_stride=31), dict(weight_row_stride=16), dict(out_row_stride=63),
               dict(residual_row_stride=63), dict(out=at["x"]), dict(out=at["weight"]),
               dict(out=at["residual"], out_row_stride=80), dict(out=at["residual"], flags=3), dict(x_row_stride=1 << 32)):
        assert call(**kw) == SHAPE, kw
    assert call(flags=8 | 1) == FLAGS
    assert call(M=0) == OK
    for kw in (dict(x=None), dict(weight=None), dict(out=None), dict(x_scale=None), dict(weight_scale=None), dict(flags=0)):
        assert call(**kw) == NULLPTR, kw                              # (flags=0: bf16 operands take no scales)
    for kw in (dict(x=at["x"] + 8), dict(weight=at["weight"] + 8), dict(x_row_stride=40), dict(weight_row_stride=40),
               dict(bias=at["bias"] + 2), dict(residual=at["residual"] + 1), dict(out=at["out"] + 1),
               dict(out=at["out"] + 2, flags=3), dict(x_scale=at["x_scale"] + 1), dict(err_flag=at["err_flag"] + 2)):
        assert call(**kw) == ALIGN, kw


@pytest.mark.parametrize("M, code", [(2 ** 31 - 1, SHAPE), (2 ** 31 - 511, SHAPE), (2 ** 31 - 512, ALIGN)])
def test_linear_rows_are_counted_in_32_bits(lib, M, code):
    # (one row fewer goes on to the next check, of a pointer that is not aligned)
    call = caller(lib, "kda_linear", L.KdaLinearArgs, dict(M=M, N=64, K=32, x=0x1000008, weight=0x2000000, out=0x3000000, x_row_stride=32,
                                                           weight_row_stride=32, out_row_stride=64))
    assert call() == code


def test_logprobs_codes(lib):
    names = ("logits", "tokens", "logprobs", "ranks", "entropy", "top_ids", "top_logprobs", "err_flag")
    at = {n: 0x100000 * (i + 1) for i, n in enumerate(names)}
    call = caller(lib, "kda_logprobs", L.KdaLogprobsArgs, dict(R=4, V=100, num_top=5, logits_row_stride=100, **at))
    for kw in (dict(R=-1), dict(R=2 ** 30), dict(V=0), dict(V=2 ** 30 + 1), dict(num_top=-1), dict(num_top=33),
               dict(logits_row_stride=99), dict(ranks=at["tokens"]), dict(top_ids=at["tokens"])):
        assert call(**kw) == SHAPE, kw
    assert call(flags=2) == FLAGS
    assert call(R=0) == OK
    for kw in (dict(logits=None), dict(entropy=None), dict(tokens=None), dict(logprobs=None), dict(ranks=None), dict(top_ids=None),
               dict(top_logprobs=None)):
        assert call(**kw) == NULLPTR, kw
    for n in names:
        assert call(**{n: at[n] + 2}) == ALIGN, n
    assert call(logits=at["logits"] + 1, flags=1) == ALIGN


@pytest.mark.parametrize("result", ["logprobs", "ranks", "entropy", "top_ids", "top_logprobs"])
def test_logprobs_keep_their_tokens(lib, result):
    names = ("logits", "tokens", "logprobs", "ranks", "entropy", "top_ids", "top_logprobs")
    at = {n: 0x100000 * (i + 1) for i, n in enumerate(names)}
    call = caller(lib, "kda_logprobs", L.KdaLogprobsArgs, dict(R=4, V=100, num_top=5, logits_row_stride=100, **at))
    assert call(**{result: at["tokens"]}) == SHAPE


def test_host_tensors_are_refused(lib):
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        kda_add_norm(z(2, 8).bfloat16(), out=z(2, 8).bfloat16())
    with pytest.raises(ValueError, match="CUDA"):
        kda_linear(z(2, 8).bfloat16(), z(4, 8).bfloat16(), z(2, 4))
    with pytest.raises(ValueError, match="CUDA"):
        kda_logprobs(z(2, 9))


@pytest.mark.parametrize("struct, field", [(L.KdaAddNormArgs, "T"), (L.KdaLinearArgs, "M"), (L.KdaLinearArgs, "N"), (L.KdaLinearArgs, "K"),
                                           (L.KdaLogprobsArgs, "R"), (L.KdaLogprobsArgs, "V")])
def test_sizes_past_32_bits_are_refused(struct, field):
    # (a tensor of 2^32 + 4 rows is none of 4)
    for n in (2 ** 31, 2 ** 32 + 4):
        with pytest.raises(ValueError, match=field):
            struct(**{field: n})
    assert getattr(struct(**{field: 2 ** 31 - 1}), field) == 2 ** 31 - 1


def test_overlaps():
    whole = torch.zeros(6, 40)
    a = whole[:, :16]
    L._apart(a, "a", whole[:, 16:], "b")                      # columns that do not meet
    L._apart(whole[:3], "a", whole[3:], "b")
    L._apart(a, "a", None, "b")
    L._apart(whole[1:4, 24:], "a", whole[:, :24], "b")
    for b in (whole[:, 15:], whole[:, :1], whole, whole[2:3], whole.view(-1)[5:9], whole[1:, :16]):
        with pytest.raises(ValueError, match="overlaps"):
            L._apart(a, "a", b, "b")
    with pytest.raises(ValueError, match="overlaps"):         # a column that runs into the next row's
        L._apart(torch.as_strided(whole, (5, 20), (40, 1), 30), "a", a, "b")


def test_reference_formulas():
    # against torch's own operators, in 64 bits
    g = torch.Generator().manual_seed(0)
    x, r, w = torch.randn(5, 64, generator=g).bfloat16(), torch.randn(5, 64, generator=g).bfloat16(), torch.rand(64, generator=g)
    h, y, s = R.add_norm(x, w, r, eps=1e-5)
    assert torch.allclose(y, torch.nn.functional.rms_norm(h, (64,), w.double(), 1e-5))
    assert torch.allclose(s * 448, y.abs().amax(-1))
    a, m, b = torch.randn(3, 16, generator=g), torch.randn(8, 16, generator=g), torch.randn(8, generator=g)
    z = torch.nn.functional.linear(a.double(), m.double(), b.double())
    for act, f in ((None, lambda v: v), ("silu", torch.nn.functional.silu), ("gelu", torch.nn.functional.gelu),
                   ("silu_gated", lambda v: torch.nn.functional.silu(v[:, :4]) * v[:, 4:])):
        assert torch.allclose(R.linear(a, m, bias=b, activation=act)[0], f(z), atol=1e-12)
    v = torch.randn(4, 50, generator=g)
    t = torch.tensor([3, -1, 49, 50], dtype=torch.int32)
    lp, ranks, ent, ids, top, _ = R.logprobs(v, t, 7)
    want = torch.log_softmax(v.double(), -1)
    assert torch.allclose(lp[[0, 2]], want[[0, 2], [3, 49]]) and lp[1] == lp[3] == 0 and ranks[1] == ranks[3] == -1
    assert torch.allclose(ent[0], torch.distributions.Categorical(logits=v[0].double()).entropy())
    assert torch.equal(ids[2], torch.topk(v[2], 7).indices.int()) and torch.allclose(top[2], torch.topk(want[2], 7).values)
