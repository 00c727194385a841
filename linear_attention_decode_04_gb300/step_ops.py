"""Python binding of the serving-step operators around the KDA layers:

- ``kda_block_tables`` (``include/kda_block_tables.h``): block tables and slot
  maps of a paged cache from the requests' lengths;
- ``kda_qk_rope`` (``include/kda_qk_rope.h``): per-head norm and rotation of q
  and k, and the write of k and v into the 8-bit cache;
- ``kda_cache_attention`` (``include/kda_cache_attention.h``): causal softmax
  attention over that cache, single tokens, multi-token steps and prompt chunks;
- ``kda_verify_draft`` (``include/kda_verify.h``): verification of the tokens
  that a multi-token decode step ran ahead with.

As in ``binding``, only arguments are marshalled here: tensors are checked
for device, dtype and layout and the C call does all the work.  Each operator
has a prepared call object (checks once, cheap to repeat, can be captured
into a CUDA graph, which must not outlive it) and a function that makes one
and runs it once.  Both run on the tensors' device whatever device is
current, on ``stream`` or that device's current stream.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import HEAD_DIM, MAX_TOKENS_PER_SEQ, KdaError, _check, _dense, _rows, kda_status_string, load_library

KDA_ROPE_INTERLEAVED = 1
BLOCK_SIZES = (16, 32, 64, 128, 256)

_i32, _i64, _u32, _f32, _ptr = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float, ctypes.c_void_p


class _Args(ctypes.Structure):
    """Base of the mirrors: whole numbers that do not fit their fields are
    refused (ctypes would keep their low bits)."""

    def __init__(self, **fields):
        for name, kind in self._fields_:
            if kind is _i32 and not -2 ** 31 <= fields.get(name, 0) < 2 ** 31:
                raise ValueError(f"{name}={fields[name]} does not fit 32 bits")
        super().__init__(**fields)


class KdaBlockTablesArgs(_Args):
    """Mirror of ``KdaBlockTablesArgs`` (field order and types must match)."""
    _fields_ = [("struct_size", _u32), ("B", _i32), ("max_blocks", _i32), ("block_size", _i32), ("num_blocks", _i32),
                ("T", _i32), ("num_free", _i32), ("cached_lens", _ptr), ("new_lens", _ptr), ("held_blocks", _ptr),
                ("held_blocks_out", _ptr), ("block_table", _ptr),
                ("block_table_stride", _i64), ("free_blocks", _ptr), ("free_head", _ptr), ("free_head_out", _ptr),
                ("cu_seqlens", _ptr), ("seq_lens", _ptr), ("positions", _ptr), ("slot_map", _ptr), ("err_flag", _ptr)]


class KdaQkRopeArgs(_Args):
    """Mirror of ``KdaQkRopeArgs``."""
    _fields_ = [("struct_size", _u32), ("T", _i32), ("num_q_heads", _i32), ("num_kv_heads", _i32),
                ("head_dim", _i32), ("rot_dim", _i32), ("block_size", _i32), ("num_blocks", _i32), ("flags", _u32),
                ("eps", _f32), ("qkv", _ptr), ("qkv_row_stride", _i64), ("q_out", _ptr), ("q_row_stride", _i64),
                ("k_out", _ptr), ("k_row_stride", _i64), ("positions", _ptr), ("freqs", _ptr), ("q_weight", _ptr),
                ("k_weight", _ptr), ("k_cache", _ptr), ("v_cache", _ptr), ("block_stride", _i64),
                ("head_stride", _i64), ("token_stride", _i64), ("k_scale", _ptr), ("v_scale", _ptr),
                ("slot_map", _ptr), ("err_flag", _ptr)]


class KdaCacheAttentionArgs(_Args):
    """Mirror of ``KdaCacheAttentionArgs``."""
    _fields_ = [("struct_size", _u32), ("B", _i32), ("T", _i32), ("num_q_heads", _i32), ("num_kv_heads", _i32),
                ("head_dim", _i32), ("block_size", _i32), ("num_blocks", _i32), ("max_blocks", _i32),
                ("max_new", _i32), ("sm_scale", _f32), ("q", _ptr), ("q_row_stride", _i64), ("out", _ptr),
                ("out_row_stride", _i64), ("cu_seqlens", _ptr), ("seq_lens", _ptr), ("block_table", _ptr),
                ("block_table_stride", _i64), ("k_cache", _ptr), ("v_cache", _ptr), ("block_stride", _i64),
                ("head_stride", _i64), ("token_stride", _i64), ("k_scale", _ptr), ("v_scale", _ptr),
                ("workspace", _ptr), ("workspace_bytes", _i64), ("err_flag", _ptr)]


class KdaVerifyArgs(_Args):
    """Mirror of ``KdaVerifyArgs``."""
    _fields_ = [("struct_size", _u32), ("N", _i32), ("T", _i32), ("V", _i32), ("draft_tokens", _ptr),
                ("target_probs", _ptr), ("target_row_stride", _i64), ("draft_probs", _ptr), ("draft_row_stride", _i64),
                ("accept_u", _ptr), ("sample_u", _ptr), ("src_slot", _ptr), ("slot_idx", _ptr), ("tokens", _ptr),
                ("num_accepted", _ptr), ("next_slot", _ptr), ("err_flag", _ptr)]


# (Looked up without asking for a device: that would initialise the driver, and a process that imports the package
# and then forks could not use CUDA in its children.)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _p(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _shaped(t, name, dtype, device, shape):
    _check(t, name, dtype, device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)} (got {tuple(t.shape)})")
    _dense(t, name)


class _Call:
    """What the prepared calls share.  ``_own`` holds the tensors that the call
    allocated.  Their memory may have held others that work on the stream they
    were made on still uses, and may hold others again once the call is
    dropped: on another stream the first run therefore waits for that stream,
    and the allocator is told of every run."""

    def _prepare(self, name: str, args: ctypes.Structure, device: torch.device, keep: tuple, own: tuple = ()):
        lib = load_library()
        self._fn = getattr(lib, name)
        self._fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
        self._fn.restype = ctypes.c_int
        self._lib, self.device, self._index = lib, device, device.index
        args.struct_size = ctypes.sizeof(args)
        self.args, self._argp = args, ctypes.addressof(args)
        self._keep, self._own = keep, own
        self._home_stream = torch.cuda.current_stream(device)
        self._home = self._home_stream.cuda_stream
        self._ordered = set()  # streams that have waited for it

    def __call__(self, stream: torch.cuda.Stream | None = None) -> None:
        # the stream's handle alone: a Stream object takes 2 us to make, which is what a small call takes on the GPU
        s = _current_raw_stream(self._index) if stream is None else stream.cuda_stream
        if s != self._home and self._own and not torch.cuda.is_current_stream_capturing():
            other = torch.cuda.current_stream(self.device) if stream is None else stream
            if s not in self._ordered:
                other.wait_stream(self._home_stream)
                self._ordered.add(s)
            for t in self._own:
                t.record_stream(other)
        if torch.cuda.current_device() == self._index:
            rc = self._fn(self._argp, s)
        else:
            with torch.cuda.device(self._index):
                rc = self._fn(self._argp, s)
        if rc != 0:
            raise KdaError(rc, f"{kda_status_string(rc)}: {self._lib.kda_last_error().decode()}")


def _err(err_flag, dev):
    if err_flag is not None:
        _check(err_flag, "err_flag", torch.int32, dev)
        if err_flag.numel() < 1:
            raise ValueError("err_flag needs one int32")


# ----------------------------------------------------------------- block tables
class KdaBlockTablesCall(_Call):
    """A prepared ``kda_block_tables`` call.  ``cached_lens`` and ``new_lens``
    int32 [B], ``block_table`` int32 [B, >= max_blocks] (rows may be strided;
    new entries are written in place), ``free_blocks`` int32 [F] with
    ``free_head`` (int32 [1] or None for 0) entries already taken.  Results
    in tensors that the call owns: ``cu_seqlens`` [B + 1], ``seq_lens`` [B],
    ``positions`` and ``slot_map`` (int64) [num_tokens], ``free_head_out``
    [1].  ``num_tokens`` is the row count of the step (the sum of the new
    lengths, or a captured step's fixed size: the rows behind get slot -1).
    ``held_blocks`` int32 [B]: the table entries that already hold blocks,
    where that may be more than the cached tokens need (a multi-token step
    whose drafts did not all stand); ``held_blocks_out`` [B] is the count
    after the call (also without ``held_blocks``)."""

    def __init__(self, cached_lens, new_lens, block_table, free_blocks, free_head=None, *, block_size: int,
                 num_blocks: int, num_tokens: int, held_blocks=None, err_flag=None):
        dev = block_table.device
        _check(block_table, "block_table", torch.int32, None)
        if block_table.dim() != 2 or block_table.shape[1] < 1 or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
            raise ValueError(f"block_table must be [B, max_blocks] with a unit inner stride (got {tuple(block_table.shape)})")
        B, M = block_table.shape
        _shaped(cached_lens, "cached_lens", torch.int32, dev, (B,))
        _shaped(new_lens, "new_lens", torch.int32, dev, (B,))
        _check(free_blocks, "free_blocks", torch.int32, dev)
        if free_blocks.dim() != 1:
            raise ValueError("free_blocks must be [F]")
        _dense(free_blocks, "free_blocks")
        if free_head is not None:
            _shaped(free_head, "free_head", torch.int32, dev, (1,))
        if held_blocks is not None:
            _shaped(held_blocks, "held_blocks", torch.int32, dev, (B,))
        _err(err_flag, dev)
        stride = block_table.stride(0) if B > 1 else max(block_table.stride(0), M)
        if stride < M:
            raise ValueError("block_table rows overlap")
        i32 = dict(dtype=torch.int32, device=dev)
        self.cu_seqlens, self.seq_lens = torch.empty(B + 1, **i32), torch.empty(B, **i32)
        self.positions = torch.empty(int(num_tokens), **i32)
        self.slot_map = torch.empty(int(num_tokens), dtype=torch.int64, device=dev)
        self.free_head_out, self.held_blocks_out = torch.empty(1, **i32), torch.empty(B, **i32)
        own = (self.cu_seqlens, self.seq_lens, self.positions, self.slot_map, self.free_head_out, self.held_blocks_out)
        args = KdaBlockTablesArgs(
            B=B, max_blocks=M, block_size=int(block_size), num_blocks=int(num_blocks), T=int(num_tokens),
            num_free=free_blocks.numel(), cached_lens=_p(cached_lens), new_lens=_p(new_lens),
            held_blocks=_p(held_blocks), held_blocks_out=_p(self.held_blocks_out),
            block_table=_p(block_table), block_table_stride=stride, free_blocks=_p(free_blocks),
            free_head=_p(free_head), free_head_out=_p(self.free_head_out), cu_seqlens=_p(self.cu_seqlens),
            seq_lens=_p(self.seq_lens), positions=_p(self.positions), slot_map=_p(self.slot_map),
            err_flag=_p(err_flag))
        self._prepare("kda_block_tables", args, dev,
                      (cached_lens, new_lens, block_table, free_blocks, free_head, held_blocks, err_flag), own)


def kda_block_tables(cached_lens, new_lens, block_table, free_blocks, free_head=None, *, block_size: int,
                     num_blocks: int, num_tokens: int, held_blocks=None, err_flag=None,
                     stream: torch.cuda.Stream | None = None):
    """Build one step's metadata on the GPU; ``block_table`` is completed in
    place.  Returns ``(cu_seqlens, seq_lens, positions, slot_map,
    free_head_out, held_blocks_out)`` as described on ``KdaBlockTablesCall``."""
    with torch.cuda.stream(stream):
        c = KdaBlockTablesCall(cached_lens, new_lens, block_table, free_blocks, free_head, block_size=block_size,
                               num_blocks=num_blocks, num_tokens=num_tokens, held_blocks=held_blocks,
                               err_flag=err_flag)
        c(stream)
    return c.cu_seqlens, c.seq_lens, c.positions, c.slot_map, c.free_head_out, c.held_blocks_out


# ------------------------------------------------------------- norm and rotation
def rope_frequencies(rot_dim: int, base: float, device=None, scaling: float = 1.0) -> torch.Tensor:
    """The ``freqs`` of ``kda_qk_rope`` for inverse frequencies base^(-2i /
    rot_dim) / scaling: turns per position as unsigned 64-bit fractions (the
    bit patterns in an int64 tensor).  Computed on the host in double
    precision and uploaded; a program keeps the result."""
    if rot_dim < 0 or rot_dim > HEAD_DIM or rot_dim % 16:
        raise ValueError(f"rot_dim must be a multiple of 16 up to {HEAD_DIM} (got {rot_dim})")
    if not (base > 0 and scaling > 0):
        raise ValueError("base and scaling must be positive")
    turns = [base ** (-2.0 * i / rot_dim) / scaling / (2 * math.pi) for i in range(rot_dim // 2)]
    bits = [round(math.ldexp(t % 1.0, 64)) % 2 ** 64 for t in turns]
    return torch.tensor([b - 2 ** 64 if b >= 2 ** 63 else b for b in bits], dtype=torch.int64, device=device)


def _cache(cache, name, dev, H):
    """Checks one cache tensor [num_blocks, H, block_size, 128] of e4m3 codes."""
    _check(cache, name, torch.float8_e4m3fn, dev)
    if cache.dim() != 4 or cache.shape[1] != H or cache.shape[3] != HEAD_DIM:
        raise ValueError(f"{name} must be [num_blocks, {H}, block_size, {HEAD_DIM}] (got {tuple(cache.shape)})")
    if cache.shape[2] not in BLOCK_SIZES:
        raise ValueError(f"{name}: block size {cache.shape[2]} is not one of {BLOCK_SIZES}")
    if cache.stride(3) != 1:
        raise ValueError(f"{name} needs a unit inner stride")


def _caches(k_cache, v_cache, k_scale, v_scale, dev, H):
    """(block size, blocks, strides) of a checked pair of caches with their scales."""
    _cache(k_cache, "k_cache", dev, H)
    _cache(v_cache, "v_cache", dev, H)
    if k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    nb, _, bs, _ = k_cache.shape
    if nb < 1:
        raise ValueError("the cache has no blocks")
    # a dimension of size one has any stride: give it the dense one
    token = k_cache.stride(2)
    head = k_cache.stride(1) if H > 1 else bs * HEAD_DIM
    block = k_cache.stride(0) if nb > 1 else H * bs * HEAD_DIM
    if token < HEAD_DIM or head < HEAD_DIM or block < HEAD_DIM or (token | head | block) % 16:
        raise ValueError(f"cache strides must be multiples of 16 and at least {HEAD_DIM} (got {k_cache.stride()})")
    _shaped(k_scale, "k_scale", torch.float32, dev, (nb, H))
    _shaped(v_scale, "v_scale", torch.float32, dev, (nb, H))
    return bs, nb, (block, head, token)


class KdaQkRopeCall(_Call):
    """A prepared ``kda_qk_rope`` call.

      qkv        bf16 [T, >= (Hq + 2 Hkv) * 128] (rows may be strided)
      positions  int32 [T]
      q_out      bf16 [T, >= Hq * 128]; may be ``qkv[:, :Hq * 128]``
      rope_freqs int64 [rot_dim / 2] from ``rope_frequencies``; None or empty
                 rotates nothing
      q_weight, k_weight  fp32 [128] or None (no norm of that part)
      k_out      bf16 [T, >= Hkv * 128] or None
      k_cache, v_cache    float8_e4m3fn [num_blocks, Hkv, block_size, 128]
                 (any order of the outer dimensions by strides), with k_scale,
                 v_scale fp32 [num_blocks, Hkv] and slot_map int64 [T] (< 0:
                 not cached); all five or none
    """

    def __init__(self, qkv, positions, q_out, *, num_q_heads: int, num_kv_heads: int, rope_freqs=None,
                 interleaved: bool = False, q_weight=None, k_weight=None, eps: float = 1e-6, k_out=None,
                 k_cache=None, v_cache=None, k_scale=None, v_scale=None, slot_map=None, err_flag=None):
        dev = qkv.device
        _check(qkv, "qkv", torch.bfloat16, None)
        Hq, Hkv = int(num_q_heads), int(num_kv_heads)
        if Hq < 1 or Hkv < 0:
            raise ValueError(f"num_q_heads={Hq}, num_kv_heads={Hkv}")
        T = qkv.shape[0] if qkv.dim() == 2 else -1
        qkv_stride = _rows(qkv, "qkv", T, (Hq + 2 * Hkv) * HEAD_DIM)
        _shaped(positions, "positions", torch.int32, dev, (T,))
        _check(q_out, "q_out", torch.bfloat16, dev)
        q_stride = _rows(q_out, "q_out", T, Hq * HEAD_DIM)
        k_stride = 0
        if k_out is not None:
            _check(k_out, "k_out", torch.bfloat16, dev)
            k_stride = _rows(k_out, "k_out", T, Hkv * HEAD_DIM)
        rot = 0
        if rope_freqs is not None and rope_freqs.numel():
            _check(rope_freqs, "rope_freqs", torch.int64, dev)
            _dense(rope_freqs, "rope_freqs")
            rot = 2 * rope_freqs.numel()
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                _shaped(w, name, torch.float32, dev, (HEAD_DIM,))
        five = (k_cache, v_cache, k_scale, v_scale, slot_map)
        cached = any(t is not None for t in five)
        bs, nb, strides = 0, 0, (0, 0, 0)
        if cached:
            if any(t is None for t in five):
                raise ValueError("k_cache, v_cache, k_scale, v_scale and slot_map go together")
            if Hkv < 1:
                raise ValueError("a cache needs num_kv_heads >= 1")
            bs, nb, strides = _caches(k_cache, v_cache, k_scale, v_scale, dev, Hkv)
            _shaped(slot_map, "slot_map", torch.int64, dev, (T,))
        _err(err_flag, dev)
        args = KdaQkRopeArgs(
            T=T, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=HEAD_DIM, rot_dim=rot, block_size=bs, num_blocks=nb,
            flags=KDA_ROPE_INTERLEAVED if interleaved else 0, eps=float(eps), qkv=_p(qkv), qkv_row_stride=qkv_stride,
            q_out=_p(q_out), q_row_stride=q_stride, k_out=_p(k_out), k_row_stride=k_stride, positions=_p(positions),
            freqs=_p(rope_freqs) if rot else None, q_weight=_p(q_weight), k_weight=_p(k_weight), k_cache=_p(k_cache),
            v_cache=_p(v_cache), block_stride=strides[0], head_stride=strides[1], token_stride=strides[2],
            k_scale=_p(k_scale), v_scale=_p(v_scale), slot_map=_p(slot_map), err_flag=_p(err_flag))
        self._prepare("kda_qk_rope", args, dev,
                      (qkv, positions, q_out, rope_freqs, q_weight, k_weight, k_out, *five, err_flag))


def kda_qk_rope(qkv, positions, q_out, *, num_q_heads: int, num_kv_heads: int, rope_freqs=None,
                interleaved: bool = False, q_weight=None, k_weight=None, eps: float = 1e-6, k_out=None, k_cache=None,
                v_cache=None, k_scale=None, v_scale=None, slot_map=None, err_flag=None,
                stream: torch.cuda.Stream | None = None) -> None:
    """Per-head norm and rotation of q and k; q to ``q_out``, k to ``k_out``
    and, with a cache, k and v into it (see ``KdaQkRopeCall``)."""
    KdaQkRopeCall(qkv, positions, q_out, num_q_heads=num_q_heads, num_kv_heads=num_kv_heads, rope_freqs=rope_freqs,
                  interleaved=interleaved, q_weight=q_weight, k_weight=k_weight, eps=eps, k_out=k_out,
                  k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale, slot_map=slot_map,
                  err_flag=err_flag)(stream)


# ------------------------------------------------------------------------ attention
def cache_attention_workspace(num_q_heads: int, num_kv_heads: int, max_new: int, device=None) -> torch.Tensor:
    """A zeroed workspace for ``kda_cache_attention`` calls with these head
    counts and at most ``max_new`` queries per sequence.  Calls ordered on one
    stream (a model's layers, captured or not) may share it; calls that may
    overlap need one each."""
    fn = load_library().kda_cache_attention_workspace_bytes
    fn.argtypes, fn.restype = [ctypes.c_int32] * 3, ctypes.c_int64
    n = fn(int(num_q_heads), int(num_kv_heads), int(max_new))
    if n < 0:
        raise ValueError(f"num_q_heads={num_q_heads} must be a positive multiple of num_kv_heads={num_kv_heads} and "
                         f"max_new={max_new} positive")
    return torch.zeros(n // 4, dtype=torch.int32, device="cuda" if device is None else device)


class KdaCacheAttentionCall(_Call):
    """A prepared ``kda_cache_attention`` call.

      q, out       bf16 [T, >= Hq * 128] (rows may be strided)
      cu_seqlens   int32 [B + 1], seq_lens int32 [B] (cached tokens, the
                   queries' own included), block_table int32 [B, max_blocks]
      k_cache, v_cache  float8_e4m3fn [num_blocks, Hkv, block_size, 128] (outer
                   dimensions in any order by strides), k_scale and v_scale
                   fp32 [num_blocks, Hkv]
      num_q_heads  Hq, a multiple of Hkv; by default q's width / 128
      max_new      the most queries a sequence has in this call (host value,
                   chooses the kernel's row tile; results are the same up to
                   rounding)
      workspace    from ``cache_attention_workspace``; by default the call
                   makes its own, and the constructor then waits for the
                   current stream once"""

    def __init__(self, q, cu_seqlens, seq_lens, block_table, k_cache, v_cache, k_scale, v_scale, out, *,
                 max_new: int = 1, num_q_heads: int | None = None, sm_scale: float = 0.0, workspace=None,
                 err_flag=None, _sync: bool = True):
        dev = q.device
        _check(q, "q", torch.bfloat16, None)
        if q.dim() != 2:
            raise ValueError(f"q must be [T, >= Hq * {HEAD_DIM}] (got {tuple(q.shape)})")
        T = q.shape[0]
        if num_q_heads is None:
            if q.shape[1] % HEAD_DIM:
                raise ValueError(f"q's width {q.shape[1]} is not a multiple of {HEAD_DIM}")
            num_q_heads = q.shape[1] // HEAD_DIM
        Hq = int(num_q_heads)
        if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
            raise ValueError(f"k_cache must be [num_blocks, Hkv, block_size, {HEAD_DIM}]")
        Hkv = k_cache.shape[1]
        if Hkv < 1 or Hq < 1 or Hq % Hkv:
            raise ValueError(f"num_q_heads={Hq} must be a positive multiple of num_kv_heads={Hkv}")
        q_stride = _rows(q, "q", T, Hq * HEAD_DIM)
        _check(out, "out", torch.bfloat16, dev)
        out_stride = _rows(out, "out", T, Hq * HEAD_DIM)
        _check(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be [B + 1]")
        _dense(cu_seqlens, "cu_seqlens")
        B = cu_seqlens.numel() - 1
        _shaped(seq_lens, "seq_lens", torch.int32, dev, (B,))
        _check(block_table, "block_table", torch.int32, dev)
        if block_table.dim() != 2 or block_table.shape[0] != B or block_table.shape[1] < 1 or \
                (block_table.shape[1] > 1 and block_table.stride(1) != 1):
            raise ValueError(f"block_table must be [{B}, max_blocks] with a unit inner stride (got {tuple(block_table.shape)})")
        M = block_table.shape[1]
        table_stride = block_table.stride(0) if B > 1 else max(block_table.stride(0), M)
        bs, nb, strides = _caches(k_cache, v_cache, k_scale, v_scale, dev, Hkv)
        _err(err_flag, dev)
        own = ()
        if workspace is None:
            workspace = cache_attention_workspace(Hq, Hkv, max_new, dev)
            own = (workspace,)
            # zeroed on the current stream, but the call may run on another
            if _sync and not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream(dev).synchronize()
        else:
            _check(workspace, "workspace", torch.int32, dev)
            _dense(workspace, "workspace")
        self.workspace = workspace
        args = KdaCacheAttentionArgs(
            B=B, T=T, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=HEAD_DIM, block_size=bs, num_blocks=nb, max_blocks=M,
            max_new=int(max_new), sm_scale=float(sm_scale), q=_p(q), q_row_stride=q_stride, out=_p(out),
            out_row_stride=out_stride, cu_seqlens=_p(cu_seqlens), seq_lens=_p(seq_lens), block_table=_p(block_table),
            block_table_stride=table_stride, k_cache=_p(k_cache), v_cache=_p(v_cache), block_stride=strides[0],
            head_stride=strides[1], token_stride=strides[2], k_scale=_p(k_scale), v_scale=_p(v_scale),
            workspace=_p(workspace), workspace_bytes=workspace.numel() * 4, err_flag=_p(err_flag))
        self._prepare("kda_cache_attention", args, dev,
                      (q, cu_seqlens, seq_lens, block_table, k_cache, v_cache, k_scale, v_scale, out, workspace,
                       err_flag), own)


def kda_cache_attention(q, cu_seqlens, seq_lens, block_table, k_cache, v_cache, k_scale, v_scale, out, *,
                        max_new: int = 1, num_q_heads: int | None = None, sm_scale: float = 0.0, workspace=None,
                        err_flag=None, stream: torch.cuda.Stream | None = None) -> None:
    """Causal attention of the batch's queries over the 8-bit paged cache, to
    ``out`` (see ``KdaCacheAttentionCall``).  Without ``workspace`` every call
    makes and clears one of 3 to 41 MB: a loop keeps one."""
    with torch.cuda.stream(stream):
        KdaCacheAttentionCall(q, cu_seqlens, seq_lens, block_table, k_cache, v_cache, k_scale, v_scale, out,
                              max_new=max_new, num_q_heads=num_q_heads, sm_scale=sm_scale, workspace=workspace,
                              err_flag=err_flag, _sync=False)(stream)


# --------------------------------------------------------------------- verification
def _prob_rows(t, name, dev, N, T):
    """[N, T, V] or [N * T, V] rows with one stride between rows: (V, stride)"""
    _check(t, name, torch.float32, dev)
    if t.dim() == 2:
        t = t.unflatten(0, (N, T)) if t.shape[0] == N * T else t
    if t.dim() != 3 or t.shape[:2] != (N, T) or t.shape[2] < 1:
        raise ValueError(f"{name} must be [{N}, {T}, V] or [{N * T}, V] (got {tuple(t.shape)})")
    V = t.shape[2]
    if V > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} needs a unit inner stride")
    row = t.stride(1) if T > 1 else t.stride(0) if N > 1 else V
    if (N > 1 and T > 1 and t.stride(0) != T * row) or row < V:
        raise ValueError(f"{name}: rows must have one stride of at least V (got strides {t.stride()})")
    return V, row


class KdaVerifyDraftCall(_Call):
    """A prepared ``kda_verify_draft`` call for N sequences of T target rows.

      draft_tokens int32 [N, T - 1]; target_probs fp32 [N, T, V] (or
      [N * T, V]); accept_u fp32 [N, T - 1] and sample_u fp32 [N], uniform in
      [0, 1); draft_probs fp32 [N, T - 1, V] or None (drafts taken as
      certain); src_slot int32 [N] or None and slot_idx int32 [N, T] or None
      as in the multi-token decode step.

    Results in tensors that the call owns: ``tokens`` [N, T] (accepted
    drafts, the sampled token, -1 behind), ``num_accepted`` [N], and with
    ``slot_idx`` ``next_slot`` [N], the next step's ``src_slot`` (else None)."""

    def __init__(self, draft_tokens, target_probs, accept_u, sample_u, *, draft_probs=None, src_slot=None,
                 slot_idx=None, err_flag=None):
        dev = target_probs.device
        _check(sample_u, "sample_u", torch.float32, None)
        _check(draft_tokens, "draft_tokens", torch.int32, dev)
        if draft_tokens.dim() != 2:
            raise ValueError("draft_tokens must be [N, T - 1]")
        N, T = draft_tokens.shape[0], draft_tokens.shape[1] + 1
        if T > MAX_TOKENS_PER_SEQ:
            raise ValueError(f"at most {MAX_TOKENS_PER_SEQ} rows per sequence (got {T})")
        _dense(draft_tokens, "draft_tokens")
        _shaped(sample_u, "sample_u", torch.float32, dev, (N,))
        _shaped(accept_u, "accept_u", torch.float32, dev, (N, T - 1))
        V, stride = _prob_rows(target_probs, "target_probs", dev, N, T)
        probs_stride = 0
        if draft_probs is not None and T > 1:
            Vd, probs_stride = _prob_rows(draft_probs, "draft_probs", dev, N, T - 1)
            if Vd != V:
                raise ValueError(f"draft_probs has {Vd} columns, target_probs {V}")
        if src_slot is not None:
            _shaped(src_slot, "src_slot", torch.int32, dev, (N,))
        self.next_slot = None
        i32 = dict(dtype=torch.int32, device=dev)
        if slot_idx is not None:
            _shaped(slot_idx, "slot_idx", torch.int32, dev, (N, T))
            self.next_slot = torch.empty(N, **i32)
        _err(err_flag, dev)
        self.tokens, self.num_accepted = torch.empty(N, T, **i32), torch.empty(N, **i32)
        drafts = T > 1
        args = KdaVerifyArgs(
            N=N, T=T, V=V, draft_tokens=_p(draft_tokens) if drafts else None, target_probs=_p(target_probs),
            target_row_stride=stride, draft_probs=_p(draft_probs) if drafts else None, draft_row_stride=probs_stride,
            accept_u=_p(accept_u) if drafts else None, sample_u=_p(sample_u), src_slot=_p(src_slot),
            slot_idx=_p(slot_idx), tokens=_p(self.tokens), num_accepted=_p(self.num_accepted),
            next_slot=_p(self.next_slot), err_flag=_p(err_flag))
        own = tuple(t for t in (self.tokens, self.num_accepted, self.next_slot) if t is not None)
        self._prepare("kda_verify_draft", args, dev,
                      (draft_tokens, target_probs, accept_u, sample_u, draft_probs, src_slot, slot_idx, err_flag), own)


def kda_verify_draft(draft_tokens, target_probs, accept_u, sample_u, *, draft_probs=None, src_slot=None,
                     slot_idx=None, err_flag=None, stream: torch.cuda.Stream | None = None):
    """Verify drafted tokens; returns ``(tokens, num_accepted, next_slot)``
    (see ``KdaVerifyDraftCall``)."""
    with torch.cuda.stream(stream):
        c = KdaVerifyDraftCall(draft_tokens, target_probs, accept_u, sample_u, draft_probs=draft_probs,
                               src_slot=src_slot, slot_idx=slot_idx, err_flag=err_flag)
        c(stream)
    return c.tokens, c.num_accepted, c.next_slot
