"""What a call may read early (weights, a decode's states) is promised not to be
written by the kernel directly ahead of it alone: it sees what an earlier one
wrote, however late that one wrote it.  And a call's own waits, which have
limits, begin when what is ahead of it has ended."""
import ctypes
import os
import subprocess

import pytest
import torch

from linear_attention_decode_04_gb300 import KdaDecodeCall, KdaLinearCall
from linear_attention_decode_04_gb300 import build as B

pytestmark = pytest.mark.gpu
LATE = 20_000_000                                  # ns, against some 10 us that the calls behind it take


@pytest.fixture(scope="module")
def late_copy(tmp_path_factory):
    """late_copy(dst, src, ns): the current stream's next kernel, whose dependents start at once, copies src to dst after ns"""
    so = str(tmp_path_factory.mktemp("late") / "liblate_writer.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "late_writer.cu")
    nv = B.nvcc()
    subprocess.run([nv, *B.ARCH, "-O2", "-shared", "-cudart", "shared", "-Xcompiler", "-fPIC", "-o", so, src, "-Xlinker",
                    f"-rpath,{B.cuda_lib_dir(nv)}"], check=True)
    fn = ctypes.CDLL(so).late_writer_copy
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p]

    def copy(dst, src, ns=LATE):
        assert dst.is_contiguous() and src.is_contiguous() and dst.nbytes == src.nbytes
        assert fn(dst.data_ptr(), src.data_ptr(), dst.nbytes, ns, torch.cuda.current_stream().cuda_stream) == 0
    return copy


def whole(g, dev, *shape):
    return torch.randint(-3, 4, shape, generator=g).bfloat16().to(dev)


# a call ahead whose CTAs leave room for those of the next one, in one tile or in several shares; then one of few rows, and pairs
@pytest.mark.parametrize("ahead", [(4, 128, 64), (4, 128, 4096), (130, 128, 256)])
@pytest.mark.parametrize("M, N, K", [(4, 256, 128), (20, 300, 2048), (300, 512, 256)])
def test_weights_written_two_kernels_ahead(ahead, M, N, K, cuda_device, late_copy):
    g, dev = torch.Generator().manual_seed(M + N), cuda_device
    a, b = whole(g, dev, ahead[0], ahead[2]), whole(g, dev, ahead[1], ahead[2])
    between = KdaLinearCall(a, b, torch.zeros(ahead[0], ahead[1], device=dev))
    x, new = whole(g, dev, M, K), whole(g, dev, N, K)
    weight, out, err = torch.zeros_like(new), torch.zeros(M, N, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    call = KdaLinearCall(x, weight, out, early_weight=True, err_flag=err)
    between()
    call()
    torch.cuda.synchronize(dev)
    assert not out.any()
    late_copy(weight, new)
    between()
    call()
    torch.cuda.synchronize(dev)
    assert torch.equal(out, x.float() @ new.float().t()) and err.item() == 0


# (the limit of a wait inside a product is 2 s) one CTA a tile, several, pairs, several pairs, many tiles
@pytest.mark.parametrize("M, N, K", [(4, 128, 64), (20, 300, 2048), (100, 2463, 5680), (300, 512, 256), (2000, 4000, 128)])
def test_kernel_ahead_takes_longer_than_a_wait_may(M, N, K, cuda_device, late_copy):
    g, dev = torch.Generator().manual_seed(M + N), cuda_device
    new, weight = whole(g, dev, M, K), whole(g, dev, N, K)
    x, out, err = torch.zeros_like(new), torch.zeros(M, N, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    call = KdaLinearCall(x, weight, out, early_weight=M < 200, err_flag=err)
    call()
    torch.cuda.synchronize(dev)
    late_copy(x, new, 2_500_000_000)
    call()
    torch.cuda.synchronize(dev)
    assert err.item() == 0 and torch.equal(out, new.float() @ weight.float().t())


def decode(N, H, T, seed, dev, early):
    """(call, its state pool, its conv windows, its results) of a decode of its own pools"""
    g = torch.Generator().manual_seed(seed)
    f = lambda *s: torch.randn(*s, generator=g).to(dev)  # noqa: E731
    HD, rows, slots = 128 * H, N * T, 1 + N * (T + 1)
    state, conv, out = f(slots, H, 128, 128) * 0.02, f(slots, 3 * HD, 3).bfloat16(), torch.zeros(rows, HD, device=dev).bfloat16()
    i32 = dict(dtype=torch.int32, device=dev)
    spec = dict(tokens_per_seq=T, src_slot=torch.arange(1, N + 1, **i32)) if T > 1 else {}
    dst = (N + 1 + torch.arange(rows, **i32)).view(N, T) if T > 1 else torch.arange(1, N + 1, **i32)
    call = KdaDecodeCall(f(rows, 3 * HD).bfloat16(), f(3, 4, HD) * 0.5, conv, state, -torch.rand(rows, H, 128, generator=g).to(dev),
                         torch.rand(rows, H, generator=g).to(dev).bfloat16(), dst, out, gate=f(rows, HD).bfloat16(),
                         norm_weight=torch.ones(128, device=dev), early_prefetch=early, **spec)
    return call, state, conv, out


@pytest.mark.parametrize("between", ["product", "decode", "multi"])
@pytest.mark.parametrize("N, H, T", [(1, 4, 1), (4, 12, 1), (3, 8, 4), (2, 4, 8)])
def test_states_written_two_kernels_ahead(N, H, T, between, cuda_device, late_copy):
    dev = cuda_device
    if between == "product":
        g = torch.Generator().manual_seed(0)
        other = KdaLinearCall(whole(g, dev, 4, 64), whole(g, dev, 128, 64), torch.zeros(4, 128, device=dev))
    else:
        other = decode(2, 6, 1 if between == "decode" else 4, 5, dev, True)[0]
    results = []
    for early in (False, True):
        call, state, conv, out = decode(N, H, T, 7, dev, early)
        new = torch.randn(state.shape, generator=torch.Generator().manual_seed(9)).to(dev)
        other()
        torch.cuda.synchronize(dev)
        late_copy(state, new)
        if not early:                              # one after another
            torch.cuda.synchronize(dev)
            assert torch.equal(state, new)
        other()
        call()
        torch.cuda.synchronize(dev)
        results.append((state, conv, out))
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_two_kernels_ahead_in_a_captured_step(cuda_device, late_copy):
    # the same order as edges of a graph: weights and states written first, a small call, then those that read them early
    g, dev = torch.Generator().manual_seed(1), cuda_device
    between = KdaLinearCall(whole(g, dev, 4, 64), whole(g, dev, 128, 64), torch.zeros(4, 128, device=dev))
    x, new = whole(g, dev, 20, 512), whole(g, dev, 300, 512)
    weight, out = torch.zeros_like(new), torch.zeros(20, 300, device=dev)
    product = KdaLinearCall(x, weight, out, early_weight=True)
    call, state, conv, y = decode(2, 4, 1, 3, dev, True)
    fresh, windows = state * 3, conv.clone()
    state.copy_(fresh)
    weight.copy_(new)
    torch.cuda.synchronize(dev)
    between()
    call()
    product()
    torch.cuda.synchronize(dev)
    want = [t.clone() for t in (state, conv, y, out)]
    assert torch.equal(out, x.float() @ new.float().t())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        late_copy(state, fresh)
        between()
        call()
        late_copy(weight, new)
        between()
        product()
    for _ in range(3):
        for t in (state, weight, y, out):
            t.zero_()
        conv.copy_(windows)
        graph.replay()
        torch.cuda.synchronize(dev)
        for a, b in zip(want, (state, conv, y, out)):
            assert torch.equal(a, b)
