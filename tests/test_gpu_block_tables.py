"""Block tables and slot maps against the 64-bit reference, bit-exact."""
import numpy as np
import pytest
import torch

import step_reference as R
from linear_attention_decode_04_gb300 import KdaBlockTablesCall, kda_block_tables

pytestmark = pytest.mark.gpu


def run(dev, cached, new, bs, *, T=None, M=None, num_blocks=None, free=None, head=0, seed=0, row_pad=0, table=None,
        with_head=True, held=None):
    rng = np.random.default_rng(seed)
    cached, new = np.asarray(cached, np.int32), np.asarray(new, np.int32)
    B = len(cached)
    need = [max(0, -(-(int(c) + int(n)) // bs)) if c >= 0 and n >= 0 else 0 for c, n in zip(cached, new)]
    M = max([1] + need) + 1 if M is None else M
    num_blocks = sum(need) + head + 20 if num_blocks is None else num_blocks
    ids = rng.permutation(num_blocks).astype(np.int32)
    if table is None:
        table = np.full((B, M), -5, np.int32)
        at = 0
        for b in range(B):
            k = min(max(-(-max(int(cached[b]), 0) // bs), 0 if held is None else held[b]), M)
            table[b, :k] = ids[at:at + k]
            at += k
        ids = ids[at:]
    free = ids if free is None else np.asarray(free, np.int32)
    T = max(0, int(np.maximum(new, 0).sum())) if T is None else T
    want = R.block_tables(cached, new, table, free, head, bs, num_blocks, T, held)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    wide = torch.full((B, M + row_pad), -77, dtype=torch.int32, device=dev)
    wide[:, :M] = t(table)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    got = kda_block_tables(t(cached), t(new), wide[:, :M], t(free), torch.tensor([head], dtype=torch.int32, device=dev)
                           if with_head else None, held_blocks=None if held is None else t(np.asarray(held, np.int32)), block_size=bs, num_blocks=num_blocks, num_tokens=T, err_flag=err)
    torch.cuda.synchronize(dev)
    assert np.array_equal(wide[:, :M].cpu().numpy(), want[0])
    assert bool((wide[:, M:] == -77).all())
    for g, w in zip(got, want[1:5]):
        assert g.cpu().tolist() == list(w)
    assert got[4].item() == want[5]
    assert got[5].cpu().tolist() == want[6]
    assert err.item() == want[7]
    return want[7]


@pytest.mark.parametrize("bs", [1, 16, 24, 64, 256])
def test_random_batches(bs, cuda_device):
    rng = np.random.default_rng(bs)
    # around the 512 rows of a CTA and the 2048 requests of a scan tile
    for B in (1, 7, 511, 513, 2047, 2048, 2049, 5000):
        new = rng.integers(0, 5, B) * (rng.random(B) < 0.9)
        new[rng.integers(0, B)] = 300
        assert run(cuda_device, rng.integers(0, 200, B), new, bs, seed=B, head=3, row_pad=2) == 0


def test_held_blocks_are_used_before_the_list(cuda_device):
    rng = np.random.default_rng(4)
    for B in (3, 600, 2500):
        cached, new = rng.integers(0, 100, B), rng.integers(0, 9, B)
        held = [-(-int(c) // 16) + int(k) for c, k in zip(cached, rng.integers(-1, 3, B))]   # too few count as enough
        assert run(cuda_device, cached, new, 16, held=held, M=12, num_blocks=20 * B + 40, seed=B) == 0
    assert run(cuda_device, [10, 20], [40, 5], 16, held=[2, 2], free=[3], num_blocks=40) == R.CAPACITY
    assert run(cuda_device, [10], [2], 16, held=[9], M=4, num_blocks=40) == 0                 # more than the row has


def test_edges(cuda_device):
    assert run(cuda_device, [], [], 16, T=5) == 0                      # no requests: only padding rows
    assert run(cuda_device, [5, 0, 16], [0, 0, 0], 16, T=0) == 0       # nothing new
    assert run(cuda_device, [0, 15, 16, 17], [1, 1, 1, 1], 16, T=700) == 0   # a padded step
    assert run(cuda_device, [0], [4000], 64, with_head=False) == 0     # one long prompt over many CTAs
    assert run(cuda_device, [0] * 3000, [1] * 3000, 16) == 0
    assert run(cuda_device, [2 ** 31 - 9], [5], 2 ** 30, M=2) == 0     # positions near 2^31


def test_errors_set_bits_and_stay_in_bounds(cuda_device):
    assert run(cuda_device, [3, -4, 5, 2 ** 31 - 2], [2, 3, -1, 9], 16) == R.SEQLENS
    assert run(cuda_device, [3, 14, 0], [20, 20, 20], 16, free=[4, 2]) == R.CAPACITY        # the list runs out
    assert run(cuda_device, [0, 0], [20, 20], 16, free=[4, 2, 1, 3], head=2) == R.CAPACITY  # it began partly used
    assert run(cuda_device, [0], [20], 16, free=[4, 2], head=7) == R.CAPACITY               # head behind the end
    assert run(cuda_device, [0], [20], 16, free=[4, 2], head=-1) == R.CAPACITY
    assert run(cuda_device, [10, 30], [40, 3], 16, M=2, num_blocks=40) == R.CAPACITY        # a row too narrow
    assert run(cuda_device, [0, 5], [9, 9], 16, T=12) == R.CAPACITY                         # more tokens than rows
    assert run(cuda_device, [0, 0], [9, 9], 16, free=[40, 1], num_blocks=40) == R.SLOT_RANGE
    assert run(cuda_device, [3], [2], 16, table=np.array([[99, 1]], np.int32), M=2, num_blocks=40) == R.SLOT_RANGE
    assert run(cuda_device, [3], [2], 16, table=np.array([[-1, 1]], np.int32), M=2, num_blocks=40) == R.SLOT_RANGE


def test_graph_replay_follows_the_lengths(cuda_device):
    dev, B, bs = cuda_device, 6, 16
    cached = torch.tensor([0, 15, 16, 40, 63, 7], dtype=torch.int32, device=dev)
    new = torch.ones(B, dtype=torch.int32, device=dev)
    table = torch.full((B, 8), -1, dtype=torch.int32, device=dev)
    table[:, :4] = torch.arange(B * 4, dtype=torch.int32, device=dev).view(B, 4)
    free = torch.arange(100, 140, dtype=torch.int32, device=dev)
    head = torch.zeros(1, dtype=torch.int32, device=dev)
    call = KdaBlockTablesCall(cached, new, table, free, head, block_size=bs, num_blocks=200, num_tokens=B)
    call()
    torch.cuda.synchronize(dev)
    g = torch.cuda.CUDAGraph()
    table[:, 4:] = -1
    with torch.cuda.graph(g):
        call()
        head.copy_(call.free_head_out)
        cached.copy_(call.seq_lens)
    c, t, h = cached.cpu().numpy().copy(), table.cpu().numpy().copy(), 0
    for _ in range(40):                                # several blocks per request, one token at a time
        g.replay()
        torch.cuda.synchronize(dev)
        t, _, lens, pos, slot, h, _, err = R.block_tables(c, [1] * B, t, free.tolist(), h, bs, 200, B)
        assert err == 0 and call.slot_map.tolist() == slot and call.positions.tolist() == pos
        assert head.item() == h and np.array_equal(table.cpu().numpy(), t)
        c = np.asarray(lens)


def steps_over_stale_tables(dev, cached, new, bs, Ts, M, free, num_blocks, head=0, held=None):
    """Calls with T = each of ``Ts`` rows on the same requests, the held blocks and the list's head of one fed to the
    next, over a table that is full of other requests' blocks.  A call's table, counts and head are those of a call with
    room for every row, and its rows the first T of that call's."""
    B, total = len(cached), sum(new)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    table = np.full((B, M), 7, np.int32)
    held = [-(-c // bs) for c in cached] if held is None else held
    g = [t(cached), t(new), torch.from_numpy(table.copy()).to(dev), t(free)]
    owners = []
    for T in Ts:
        want = R.block_tables(cached, new, table, free, head, bs, num_blocks, max(T, total), held)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        got = kda_block_tables(*g, t([head]), held_blocks=t(held), block_size=bs, num_blocks=num_blocks, num_tokens=T,
                               err_flag=err)
        assert err.item() == want[7] | (R.CAPACITY if T < total else 0)
        table, head, held = want[0], want[5], want[6]
        assert np.array_equal(g[2].cpu().numpy(), table)
        assert got[0].tolist() == want[1] and got[1].tolist() == want[2]
        assert got[2].tolist() == want[3][:T] and got[3].tolist() == want[4][:T]
        assert got[4].item() == head and got[5].tolist() == held
        owners = got[3].tolist()
    return owners


def test_blocks_for_rows_past_the_end_are_in_the_table(cuda_device):
    # a step with more tokens than rows, then the same requests with room for all: the blocks that the first took and
    # counted as held are the ones that the second uses, not what the table held before
    slots = steps_over_stale_tables(cuda_device, [0, 0], [16, 16], 16, [16, 32], 3, list(range(20, 30)), 40)
    assert slots == [*range(20 * 16, 21 * 16), *range(21 * 16, 22 * 16)]
    # requests cut in the middle and past the end, several blocks each, rows of no CTA; a list that runs out or names
    # blocks that are not there
    steps_over_stale_tables(cuda_device, [3, 0, 40, 15], [90, 0, 33, 600], 16, [0, 50, 95, 1000], 45, list(range(8, 99)), 100)
    steps_over_stale_tables(cuda_device, [0, 5, 0], [40, 70, 64], 16, [41, 60, 200], 6, [9, 10, 11, 12, 13], 20)
    steps_over_stale_tables(cuda_device, [0, 0], [20, 60], 16, [10, 80], 5, [9, 55, 10, -3, 11, 12], 20)
    # tables that are too narrow, blocks held from an earlier step, batches over several tiles of the scan
    steps_over_stale_tables(cuda_device, [0, 10], [100, 100], 24, [30, 200], 3, list(range(50)), 50, held=[1, 2])
    rng = np.random.default_rng(11)
    cached, new = rng.integers(0, 60, 2500).tolist(), rng.integers(0, 40, 2500).tolist()
    steps_over_stale_tables(cuda_device, cached, new, 16, [700, sum(new) // 2, sum(new)], 8, list(range(20000)), 20000, head=5)
