"""What a call may read early (weights, a decode's states) is promised not to be
written by the kernel directly ahead of it alone: it sees what an earlier one
wrote, however late that one wrote it."""
import ctypes
import os
import subprocess

import pytest
import torch

from linear_attention_decode_04_gb300 import KdaLinearCall, kda_linear
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
