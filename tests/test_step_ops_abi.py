"""The serving-step operators on the host: struct mirrors, argument codes of
the C ABI (before any CUDA call, with pointers that are never dereferenced),
refusals of the Python calls, and the rotation's phase table."""
import ctypes
import math
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import step_reference as R
from linear_attention_decode_04_gb300 import binding, kda_block_tables, kda_qk_rope, kda_verify_draft, rope_frequencies
from linear_attention_decode_04_gb300 import build as B
from linear_attention_decode_04_gb300 import step_ops as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULLPTR, SHAPE, ALIGN, FLAGS, ABI = 0, -1, -2, -3, -4, -6


@pytest.fixture(scope="module")
def lib():
    B.build()
    return binding.load_library()


def header_fields(header, name):
    text = open(os.path.join(ROOT, "include", header)).read()
    body = text[text.index(f"typedef struct {name} {{") + len(f"typedef struct {name} {{"):text.index(f"}} {name};")]
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    out = []
    for decl in re.findall(r"([^;]+);", body):
        first, *rest = decl.split(",")
        out += [first.split()[-1].lstrip("*")] + [r.strip().lstrip("*") for r in rest]
    return out


@pytest.mark.parametrize("header, struct", [("kda_block_tables.h", S.KdaBlockTablesArgs),
                                            ("kda_qk_rope.h", S.KdaQkRopeArgs), ("kda_verify.h", S.KdaVerifyArgs),
                                            ("kda_cache_attention.h", S.KdaCacheAttentionArgs)])
def test_struct_mirrors(header, struct):
    assert header_fields(header, struct.__name__) == [f for f, _ in struct._fields_]


def caller(lib, name, cls, good):
    fn = getattr(lib, name)
    fn.argtypes, fn.restype = [ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int

    def call(**kw):
        a = cls(struct_size=ctypes.sizeof(cls))
        for k, v in {**good, **kw}.items():
            setattr(a, k, v)
        return fn(ctypes.addressof(a), None)
    assert fn(None, None) == NULLPTR
    assert call(struct_size=8) == ABI
    return call


def test_block_tables_codes(lib):
    names = ("cached_lens", "new_lens", "block_table", "free_blocks", "free_head", "free_head_out", "cu_seqlens",
             "seq_lens", "positions", "slot_map")
    call = caller(lib, "kda_block_tables", S.KdaBlockTablesArgs,
                  dict(B=4, max_blocks=8, block_size=16, num_blocks=32, T=9, num_free=12, block_table_stride=8,
                       **{n: 0x10000 * (i + 1) for i, n in enumerate(names)}))
    for kw in (dict(B=-1), dict(max_blocks=0), dict(block_size=0), dict(num_blocks=0), dict(T=-1), dict(num_free=-1),
               dict(block_table_stride=7), dict(free_head=0x60000)):
        assert call(**kw) == SHAPE, kw
    for n in set(names) - {"free_head"}:
        assert call(**{n: None}) == NULLPTR, n
    for n in names:
        assert call(**{n: 0x10002}) == ALIGN, n
    assert call(slot_map=0x10004) == ALIGN


def test_qk_rope_codes(lib):
    names = ("qkv", "q_out", "positions", "freqs", "q_weight", "k_weight", "k_cache", "v_cache", "k_scale", "v_scale",
             "slot_map")
    call = caller(lib, "kda_qk_rope", S.KdaQkRopeArgs,
                  dict(T=4, num_q_heads=4, num_kv_heads=2, head_dim=128, rot_dim=64, block_size=16, num_blocks=8,
                       qkv_row_stride=1024, q_row_stride=512, k_row_stride=256, block_stride=2 * 16 * 128,
                       head_stride=2048, token_stride=128,
                       **{n: 0x10000 * (i + 1) for i, n in enumerate(names)}))
    for kw in (dict(head_dim=64), dict(T=-1), dict(num_q_heads=0), dict(rot_dim=8), dict(rot_dim=144),
               dict(block_size=24), dict(block_size=512), dict(num_blocks=0), dict(qkv_row_stride=1016),
               dict(q_row_stride=504), dict(k_out=0x200000, k_row_stride=128), dict(token_stride=64),
               dict(k_out=0x10000 + 4 * 256)):
        assert call(**kw) == SHAPE, kw
    assert call(flags=2) == FLAGS
    assert call(T=0) == OK
    for n in ("qkv", "q_out", "positions", "freqs", "k_cache", "v_scale", "slot_map"):
        assert call(**{n: None}) == NULLPTR, n
    for kw in (dict(qkv=0x10008), dict(q_out=0x10008), dict(qkv_row_stride=1028), dict(token_stride=136),
               dict(slot_map=0x10004), dict(q_weight=0x10004), dict(k_cache=0x10008), dict(positions=0x10002)):
        assert call(**kw) == ALIGN, kw


def test_cache_attention_codes(lib):
    names = ("q", "out", "cu_seqlens", "seq_lens", "block_table", "k_cache", "v_cache", "k_scale", "v_scale", "workspace")
    size = lib.kda_cache_attention_workspace_bytes
    size.argtypes, size.restype = [ctypes.c_int32] * 3, ctypes.c_int64
    call = caller(lib, "kda_cache_attention", S.KdaCacheAttentionArgs,
                  dict(B=3, T=7, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=32, num_blocks=9, max_blocks=4,
                       max_new=3, q_row_stride=1024, out_row_stride=1024, block_table_stride=4, block_stride=8192,
                       head_stride=4096, token_stride=128, workspace_bytes=size(8, 2, 3),
                       **{n: 0x10000 * (i + 1) for i, n in enumerate(names)}))
    for kw in (dict(head_dim=64), dict(B=-1), dict(T=-1), dict(num_q_heads=7), dict(num_kv_heads=0), dict(block_size=8),
               dict(block_size=48), dict(num_blocks=0), dict(max_blocks=0), dict(max_new=0), dict(q_row_stride=1016),
               dict(out_row_stride=512), dict(block_table_stride=3), dict(token_stride=64), dict(head_stride=0),
               dict(workspace_bytes=size(8, 2, 3) - 1), dict(T=2 ** 30)):
        assert call(**kw) == SHAPE, kw
    assert call(B=0) == OK and call(T=0) == OK
    for n in names:
        assert call(**{n: None}) == NULLPTR, n
    for kw in (dict(q=0x10008), dict(out=0x10008), dict(q_row_stride=1028), dict(k_cache=0x10008), dict(v_cache=0x10004),
               dict(token_stride=136), dict(workspace=0x10008), dict(k_scale=0x10002), dict(cu_seqlens=0x10002)):
        assert call(**kw) == ALIGN, kw
    assert size(8, 2, 3) > 4096 and size(96, 8, 8) > size(8, 2, 3)
    assert size(8, 3, 1) == size(0, 1, 1) == size(8, 2, 0) == -1


def test_verify_codes(lib):
    names = ("draft_tokens", "target_probs", "draft_probs", "accept_u", "sample_u", "src_slot", "slot_idx", "tokens",
             "num_accepted", "next_slot")
    call = caller(lib, "kda_verify_draft", S.KdaVerifyArgs,
                  dict(N=4, T=3, V=100, target_row_stride=100, draft_row_stride=100,
                       **{n: 0x10000 * (i + 1) for i, n in enumerate(names)}))
    for kw in (dict(N=-1), dict(T=0), dict(T=9), dict(V=0), dict(target_row_stride=99), dict(draft_row_stride=99),
               dict(N=2 ** 30)):
        assert call(**kw) == SHAPE, kw
    assert call(N=0) == OK
    for n in set(names) - {"draft_probs", "src_slot"}:
        assert call(**{n: None}) == NULLPTR, n
    for n in names:
        assert call(**{n: 0x10002}) == ALIGN, n


def test_results_in_the_place_of_inputs(lib):
    # refused before any CUDA call; which places are allowed is tested on the GPU
    names = ("cached_lens", "new_lens", "held_blocks", "free_blocks", "free_head", "free_head_out", "block_table",
             "cu_seqlens", "seq_lens", "positions", "held_blocks_out", "slot_map")
    at = {n: 0x10000 * (i + 1) for i, n in enumerate(names)}
    call = caller(lib, "kda_block_tables", S.KdaBlockTablesArgs,
                  dict(B=4, max_blocks=8, block_size=16, num_blocks=32, T=9, num_free=12, block_table_stride=8, **at))
    for out, given in (("seq_lens", "cached_lens"), ("seq_lens", "new_lens"), ("held_blocks_out", "cached_lens"),
                       ("held_blocks_out", "held_blocks"), ("cu_seqlens", "new_lens"), ("positions", "cached_lens"),
                       ("free_head_out", "free_head"), ("block_table", "free_blocks")):
        assert call(**{out: at[given]}) == SHAPE, out
    names = ("qkv", "q_out", "positions", "freqs")
    at = {n: 0x10000 * (i + 1) for i, n in enumerate(names)}
    call = caller(lib, "kda_qk_rope", S.KdaQkRopeArgs,
                  dict(T=4, num_q_heads=4, num_kv_heads=2, head_dim=128, rot_dim=64, qkv_row_stride=1024,
                       q_row_stride=512, k_row_stride=256, **at))
    assert call(q_out=at["qkv"]) == SHAPE
    assert call(k_out=at["qkv"] + 4 * 256) == SHAPE
    names = ("q", "out", "cu_seqlens", "seq_lens", "block_table", "k_cache", "v_cache", "k_scale", "v_scale", "workspace")
    call = caller(lib, "kda_cache_attention", S.KdaCacheAttentionArgs,
                  dict(B=3, T=7, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=32, num_blocks=9, max_blocks=4,
                       max_new=1, q_row_stride=1024, out_row_stride=1024, block_table_stride=4, block_stride=8192,
                       head_stride=4096, token_stride=128, workspace_bytes=1 << 30,
                       **{n: 0x10000 * (i + 1) for i, n in enumerate(names)}))
    assert call(out=0x10000) == SHAPE
    names = ("draft_tokens", "target_probs", "accept_u", "sample_u", "src_slot", "slot_idx", "tokens", "num_accepted",
             "next_slot")
    at = {n: 0x10000 * (i + 1) for i, n in enumerate(names)}
    call = caller(lib, "kda_verify_draft", S.KdaVerifyArgs, dict(N=4, T=3, V=100, target_row_stride=100, **at))
    for out, given in (("tokens", "draft_tokens"), ("next_slot", "slot_idx"), ("num_accepted", "src_slot")):
        assert call(**{out: at[given]}) == SHAPE, out


def test_host_tensors_are_refused(lib):
    i32, f32 = dict(dtype=torch.int32), dict(dtype=torch.float32)
    with pytest.raises(ValueError, match="CUDA"):
        kda_block_tables(torch.zeros(2, **i32), torch.zeros(2, **i32), torch.zeros(2, 3, **i32), torch.zeros(4, **i32),
                         block_size=16, num_blocks=4, num_tokens=2)
    with pytest.raises(ValueError, match="CUDA"):
        kda_qk_rope(torch.zeros(2, 512, dtype=torch.bfloat16), torch.zeros(2, **i32),
                    torch.zeros(2, 256, dtype=torch.bfloat16), num_q_heads=2, num_kv_heads=1)
    with pytest.raises(ValueError, match="CUDA"):
        kda_verify_draft(torch.zeros(2, 1, **i32), torch.zeros(2, 2, 9, **f32), torch.zeros(2, 1, **f32),
                         torch.zeros(2, **f32))


def test_rope_frequencies():
    for rot, base, scaling in ((128, 1e4, 1.0), (64, 1e6, 1.0), (16, 5e5, 8.0)):
        f = [int(v) % 2 ** 64 for v in rope_frequencies(rot, base, scaling=scaling).tolist()]
        assert len(f) == rot // 2
        for pos in (0, 1, 4097, 10 ** 6, 2 ** 31 - 1):
            for i, v in enumerate(f):
                # the angle in turns modulo one against a long division: freqs hold double precision, so a position
                # near 2^31 costs at most 2^31 * 2^-54 turns
                turns = pos * (base ** (-2.0 * i / rot) / scaling) / (2 * math.pi)
                d = (pos * v % 2 ** 64) / 2.0 ** 64 - math.fmod(turns, 1.0)
                assert abs(d - round(d)) < 2.0 ** -20
    assert rope_frequencies(0, 1e4).numel() == 0
    for bad in (8, 144, -16):
        with pytest.raises(ValueError):
            rope_frequencies(bad, 1e4)
    with pytest.raises(ValueError):
        rope_frequencies(64, 0.0)


def test_reference_rounds_like_torch():
    # the references' brute-force e4m3 rounding against torch's, within range
    x = np.concatenate([np.linspace(-460, 460, 4001), 2.0 ** np.linspace(-14, 8, 400), [0.0, -0.0, np.nan]])
    want = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = R.e4m3_nearest(x.astype(np.float32).astype(np.float64))
    assert np.array_equal(got[:-1], want[:-1]) and got[-1] & 127 == 127


def test_attention_workspace_grows_with_max_new(lib):
    size = lib.kda_cache_attention_workspace_bytes
    size.argtypes, size.restype = [ctypes.c_int32] * 3, ctypes.c_int64
    for G in (1, 3, 8, 50):
        sizes = [size(2 * G, 2, n) for n in range(1, 300)]
        assert sizes == sorted(sizes) and sizes[-1] < 2 ** 26


def test_import_leaves_cuda_to_forked_children():
    # a server imports the package and then forks workers that use CUDA: importing must not initialise the driver, which
    # marks every later fork as unable to.  A process of its own, so that no other test's use of CUDA counts.
    code = ("import os, sys, torch\n"
            "import linear_attention_decode_04_gb300\n"
            "assert not torch.cuda.is_initialized()\n"
            "pid = os.fork()\n"
            "if pid == 0:\n"
            "    os._exit(3 if torch.cuda._is_in_bad_fork() else 0)\n"
            "sys.exit(os.waitstatus_to_exitcode(os.waitpid(pid, 0)[1]))\n")
    assert subprocess.run([sys.executable, "-c", code], cwd=ROOT, timeout=300).returncode == 0
