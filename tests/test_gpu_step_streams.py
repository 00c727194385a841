"""Prepared serving-step calls on another stream than the one they were made
on: the memory of their results may have held tensors that work queued on
that stream still writes."""
import numpy as np
import pytest
import torch

import step_reference as R
from linear_attention_decode_04_gb300 import KdaBlockTablesCall, KdaVerifyDraftCall

pytestmark = pytest.mark.gpu


def results_in_used_memory(make, results):
    """Runs ``make()``'s call on a side stream while the current one still writes tensors that were dropped, into whose
    memory the call's results went.  Returns the call, finished."""
    dev = torch.device("cuda", torch.cuda.current_device())
    side = torch.cuda.Stream(dev)
    used = [torch.empty(128, dtype=torch.int32, device=dev) for _ in range(256)]
    torch.cuda.synchronize(dev)
    torch.cuda._sleep(200_000_000)                      # some 0.1 s
    for u in used:
        u.fill_(77)
    at = {u.data_ptr() for u in used}
    del used, u
    call = make()
    assert any(t.data_ptr() in at for t in results(call))
    call(side)
    call(side)
    torch.cuda.synchronize(dev)
    return call


def test_verification_results(cuda_device):
    rng = np.random.default_rng(3)
    p = rng.random((5, 3, 60), np.float32)
    p /= p.sum(-1, keepdims=True)
    draft, u, su = rng.integers(0, 60, (5, 2)).astype(np.int32), rng.random((5, 2), np.float32), rng.random(5, np.float32)
    g = [torch.from_numpy(a).to(cuda_device) for a in (draft, p, u, su)]
    call = results_in_used_memory(lambda: KdaVerifyDraftCall(*g), lambda c: (c.tokens, c.num_accepted))
    want = R.verify(draft, p, u, su)
    assert call.tokens.tolist() == want[0] and call.num_accepted.tolist() == want[1]


def test_block_table_results(cuda_device):
    i = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda_device)  # noqa: E731
    cached, new = [3, 0, 40], [2, 1, 17]
    table = np.full((3, 5), -1, np.int32)
    table[0, 0], table[2, :3] = 9, [4, 5, 6]
    free = [20, 21, 22, 23]
    g = (i(cached), i(new), torch.from_numpy(table).to(cuda_device), i(free))
    want = R.block_tables(cached, new, table, free, 0, 16, 30, 20)
    call = results_in_used_memory(lambda: KdaBlockTablesCall(*g, block_size=16, num_blocks=30, num_tokens=20),
                                  lambda c: (c.cu_seqlens, c.seq_lens, c.positions, c.slot_map))
    assert np.array_equal(g[2].cpu().numpy(), want[0])
    assert call.cu_seqlens.tolist() == want[1] and call.seq_lens.tolist() == want[2]
    assert call.positions.tolist() == want[3] and call.slot_map.tolist() == want[4]
    assert call.free_head_out.item() == want[5] and call.held_blocks_out.tolist() == want[6]
