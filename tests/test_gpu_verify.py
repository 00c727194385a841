"""Verification of drafted tokens against exact integer arithmetic: the
results are whole numbers and have to be equal."""
import numpy as np
import pytest
import torch

import step_reference as R
from linear_attention_decode_04_gb300 import KdaVerifyDraftCall, kda_verify_draft

pytestmark = pytest.mark.gpu


def inputs(N, T, V, seed, probs=True, near=0.6):
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(N, T, V)) * 3

    def softmax(x):
        e = np.exp(x - x.max(-1, keepdims=True))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)
    p, q = softmax(z), softmax(z[:, :T - 1] + near * rng.normal(size=(N, T - 1, V)))
    draft = np.array([[rng.choice(V, p=q[n, t] / q[n, t].astype(np.float64).sum()) if probs else int(p[n, t].argmax())
                       for t in range(T - 1)] for n in range(N)], np.int32).reshape(N, T - 1)
    return dict(draft=draft, p=p, u=rng.random((N, T - 1), np.float32), su=rng.random(N, np.float32),
                q=q if probs else None, src=None,
                slots=(rng.permutation(N * T) + 1).astype(np.int32).reshape(N, T))


def check(dev, x, row_pad=0, flat=False):
    t = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731

    def rows(a):
        if a is None or not row_pad:
            return t(a)
        wide = torch.full((*a.shape[:2], a.shape[2] + row_pad), 9.0, device=dev)
        wide[..., :a.shape[2]] = t(a)
        return wide[..., :a.shape[2]]
    p = rows(x["p"])
    if flat:
        p = p.reshape(-1, p.shape[-1])
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    tok, acc, nxt = kda_verify_draft(t(x["draft"]), p, t(x["u"]), t(x["su"]), draft_probs=rows(x["q"]),
                                     src_slot=t(x["src"]), slot_idx=t(x["slots"]), err_flag=err)
    want = R.verify(x["draft"], x["p"], x["u"], x["su"], x["q"], x["src"], x["slots"])
    assert acc.tolist() == want[1]
    assert tok.tolist() == want[0]
    if x["slots"] is not None:
        assert nxt.tolist() == want[2]
    assert err.item() == want[3]
    return want


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("N, T, V", [(1, 1, 1), (1, 4, 5), (3, 8, 127), (5, 2, 128), (4, 4, 1000), (2, 3, 16384),
                                     (2, 4, 50001), (80, 3, 300), (160, 3, 300), (310, 2, 129), (700, 2, 64)])
def test_matches_exact_arithmetic(N, T, V, probs, cuda_device):
    # every cluster size (by N), parts that end inside a warp's range, unaligned rows (odd V)
    # (of batches whose rows are short where N is large: test_large_batches_of_long_rows has the others)
    check(cuda_device, inputs(N, T, V, N + T + V, probs))


def test_row_strides_and_flat_rows(cuda_device):
    x = inputs(4, 3, 501, 5)
    check(cuda_device, x, row_pad=3)       # rows on no 16-byte boundary
    check(cuda_device, x, row_pad=11)      # 512 floats apart: aligned rows, ragged end
    check(cuda_device, x, flat=True)


def test_accept_and_refuse_edges(cuda_device):
    x = inputs(6, 4, 200, 7)
    x["u"][0] = 0.0                                  # everything with mass is accepted
    x["q"][1] = x["p"][1, :3]                        # q = p: accepted for every u < 1
    x["u"][2] = np.nextafter(np.float32(1), np.float32(0))
    x["q"][3] = x["p"][3, :3]                        # q = p and u = 1: refused, and no residual mass: p itself
    x["u"][3] = 1.0
    x["p"][4, 0, x["draft"][4, 0]] = 0.0             # no target mass: refused even with u = 0
    x["u"][4] = 0.0
    x["p"][5, 0] = 0.0                               # a row without any mass
    w = check(cuda_device, x)
    assert w[1][1] == 3 and w[1][3] == 0 and w[1][4] == 0 and w[0][5][0] == 199


def test_border_values_of_the_uniform(cuda_device):
    # point masses: the running sum meets the goal exactly
    p = np.zeros((8, 1, 64), np.float32)
    p[:, 0, [3, 17, 40, 63]] = 0.25
    su = np.array([0.0, 0.25, 0.5, 0.75, np.nextafter(np.float32(0.25), np.float32(0)),
                   np.nextafter(np.float32(1), np.float32(0)), 1.0, np.nan], np.float32)
    x = dict(draft=np.zeros((8, 0), np.int32), p=p, u=np.zeros((8, 0), np.float32), su=su, q=None, src=None, slots=None)
    w = check(cuda_device, x)
    assert [t[0] for t in w[0]] == [3, 17, 40, 63, 3, 63, 63, 3]


def test_invalid_probabilities_count_as_nothing(cuda_device):
    x = inputs(4, 2, 300, 11)
    x["p"][0, :, 10:200] = np.nan
    x["p"][1, :, ::3] = -1.0
    x["p"][2, :, 7] = 5.0                            # above one counts as one
    x["q"][3, :, 5] = np.nan
    check(cuda_device, x)


def test_padding_absent_and_bad_drafts(cuda_device):
    x = inputs(7, 4, 150, 13)
    x["src"] = np.array([3, 0, 5, -2, 1, 2, 9], np.int32)
    x["u"][:] = 0.0
    x["draft"][0, 1] = -1                            # one draft only
    x["draft"][2, 0] = -1                            # none
    x["draft"][4, 2] = 150                           # out of the vocabulary
    w = check(cuda_device, x)
    assert w[1][0] == 1 and w[1][1] == 0 and w[1][2] == 0 and w[1][4] == 2 and w[3] == R.TOKEN_RANGE


def test_padding_rows_are_not_read(cuda_device):
    # the padding sequence's rows hold NaN and its drafts nonsense; the others are unaffected
    x = inputs(3, 3, 90, 17)
    x["src"] = np.array([1, 0, 2], np.int32)
    x["p"][1] = np.nan
    x["draft"][1] = 77777
    y = {k: (None if v is None else v.copy()) for k, v in x.items()}
    y["draft"][1] = 0                                # the reference does not look at it either
    assert R.verify(*(x[k] for k in ("draft", "p", "u", "su", "q", "src", "slots")))[3] == 0
    check(cuda_device, x)


def test_graph_and_side_stream(cuda_device):
    dev = cuda_device
    x, y = inputs(5, 4, 700, 19), inputs(5, 4, 700, 23)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    d, p, u, su, q, sl = (t(x[k]) for k in ("draft", "p", "u", "su", "q", "slots"))
    call = KdaVerifyDraftCall(d, p, u, su, draft_probs=q, slot_idx=sl)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    call(side)
    side.synchronize()
    assert call.tokens.tolist() == R.verify(*(x[k] for k in ("draft", "p", "u", "su", "q", "src", "slots")))[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for dst, k in ((d, "draft"), (p, "p"), (u, "u"), (su, "su"), (q, "q"), (sl, "slots")):
        dst.copy_(t(y[k]))
    g.replay()
    want = R.verify(*(y[k] for k in ("draft", "p", "u", "su", "q", "src", "slots")))
    assert call.tokens.tolist() == want[0] and call.next_slot.tolist() == want[2]


def test_refusals(cuda_device):
    t = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=cuda_device)  # noqa: E731
    d, p, u, su = t(2, 3, dt=torch.int32), t(2, 4, 9), t(2, 3), t(2)
    kda_verify_draft(d, p, u, su)
    for bad in (lambda: kda_verify_draft(d.long(), p, u, su), lambda: kda_verify_draft(d, p.double(), u, su),
                lambda: kda_verify_draft(d, p, u[:, :2], su)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(ValueError, match="at most"):
        kda_verify_draft(t(2, 8, dt=torch.int32), t(2, 9, 9), t(2, 8), su)
    with pytest.raises(ValueError, match="columns"):
        kda_verify_draft(d, p, u, su, draft_probs=t(2, 3, 8))
    with pytest.raises(ValueError, match="stride"):
        kda_verify_draft(d, t(2, 5, 9)[:, :4], u, su)


@pytest.mark.parametrize("V", [7, 9, 130, 2048, 5000, 40000])
@pytest.mark.parametrize("value", [1.0, 0.5, float("inf")])
def test_rows_that_sum_to_more_still_give_a_token(value, V, cuda_device):
    # softmax outputs by mistake unnormalised: which token is not defined, but one in range is written
    N, T = 6, 2
    p = torch.full((N, T, V), value, device=cuda_device)
    draft = torch.full((N, 1), -1, dtype=torch.int32, device=cuda_device)
    u = torch.zeros(N, 1, device=cuda_device)
    su = torch.linspace(0, 1, N, device=cuda_device)
    call = KdaVerifyDraftCall(draft, p, u, su)
    call.tokens.fill_(-7)
    call()
    tok = call.tokens.cpu()
    assert ((tok[:, 0] >= 0) & (tok[:, 0] < V)).all() and (tok[:, 1] == -1).all()


@pytest.mark.parametrize("N, V", [(3, 40000), (400, 300)])
def test_next_slot_in_the_place_of_src_slot(N, V, cuda_device):
    # a captured loop keeps one array of slots; several CTAs a sequence, and one
    x = inputs(N, 3, V, 5)
    x["src"] = (np.arange(N) % 3).astype(np.int32)          # every third one is padding
    want = R.verify(x["draft"], x["p"], x["u"], x["su"], x["q"], x["src"], x["slots"])
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda_device)  # noqa: E731
    src = t(x["src"])
    call = KdaVerifyDraftCall(t(x["draft"]), t(x["p"]), t(x["u"]), t(x["su"]), draft_probs=t(x["q"]), src_slot=src,
                              slot_idx=t(x["slots"]))
    call.args.next_slot = src.data_ptr()
    call()
    assert src.tolist() == want[2] and call.num_accepted.tolist() == want[1] and call.tokens.tolist() == want[0]


class SharedRows:
    """[n, t] rows that are rows of a small pool, read as an array by the reference."""

    def __init__(self, pool, at):
        self.pool, self.at, self.shape = pool, at, (*at.shape, pool.shape[1])

    def __getitem__(self, i):
        row = self.pool[self.at[i[0], i[1]]]
        return row if len(i) == 2 else row[i[2]]


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("N, T, V, cluster", [(39, 2, 140001, 8), (80, 3, 140001, 8), (256, 4, 131072, 4), (310, 2, 40001, 2),
                                              (700, 2, 16385, 1)])
def test_large_batches_of_long_rows(N, T, V, cluster, probs, cuda_device):
    # batches of more sequences than the 512-thread kernel takes, whose rows are long: clusters are made larger again
    # (CTAs per sequence: the rule of the launch, repeated here), and a warp's part takes many trips
    c = 8
    while c > 1 and N * c > 4 * 152:
        c //= 2
    while c < 8 and V // (2 * c) > 16384:
        c *= 2
    assert N * 8 > 2 * 152 and c == cluster
    rng = np.random.default_rng(N + T + V)
    z = rng.normal(size=(7, V)) * 3

    def softmax(x):
        e = np.exp(x - x.max(-1, keepdims=True))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)
    pool, near = softmax(z), softmax(z + 0.6 * rng.normal(size=z.shape))
    at = rng.integers(0, 7, (N, T))
    # drafts from the draft model's rows by inversion; without them, the target's likely tokens
    cum = np.cumsum((near if probs else pool).astype(np.float64), -1)
    draft = np.array([[min(int(np.searchsorted(cum[at[n, t]], rng.random())), V - 1) for t in range(T - 1)]
                      for n in range(N)], np.int32)
    u, su = rng.random((N, T - 1), np.float32) * np.float32(1.0 if probs else 2e-3), rng.random(N, np.float32)
    slots = (rng.permutation(N * T) + 1).astype(np.int32).reshape(N, T)
    want = R.verify(draft, SharedRows(pool, at), u, su, SharedRows(near, at[:, :-1]) if probs else None, None, slots)
    g = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda_device)  # noqa: E731
    rows = g(at)
    tok, acc, nxt = kda_verify_draft(g(draft), g(pool)[rows], g(u), g(su), slot_idx=g(slots),
                                     draft_probs=g(near)[rows[:, :-1]] if probs else None)
    assert acc.tolist() == want[1] and tok.tolist() == want[0] and nxt.tolist() == want[2]
    assert 0 < sum(want[1]) < N * (T - 1)               # drafts of both kinds were met
