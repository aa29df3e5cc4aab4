"""What the 4-bit cache's binding and entries take and refuse besides shapes (no GPU needed)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import sparse_quantized_attention_gb300 as ffd
from tests.test_kv4_host import FAKE, OnGpu, lib, rows_call  # noqa: F401  (lib is a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("read", [False, True], ids=["write", "read"])
def test_no_rows_without_storage(lib, read):
    """An empty tensor has no address: rows of which there are none may be NULL."""
    assert torch.empty((0, 2, 128), dtype=torch.bfloat16).data_ptr() == 0
    assert rows_call(lib, read, total=0, k=None, v=None) == 0
    assert rows_call(lib, read, total=0, cu=None, k=None, v=None) == 0
    assert rows_call(lib, read, total=0, v=None) == 0
    assert rows_call(lib, read, total=6, k=None, v=None) == 1
    # the other arguments are looked at all the same
    assert rows_call(lib, read, total=0, k=None, v=None, pos=None) == 1
    assert rows_call(lib, read, total=0, k=None, v=None, desc=(4, 2, 64, 64)) == 2
    assert rows_call(lib, read, total=0, k=None, v=None, dtype=2) == 1


@pytest.mark.parametrize("read", [False, True], ids=["write", "read"])
def test_error_word(lib, read):
    """A kernel adds to four bytes at it: it has to be aligned and as large."""
    d = ctypes.byref(ffd.CacheDesc(4, 2, 128, 64))

    def call(err):  # of no rows: nothing is launched when all is well
        if read:
            return lib.ffd_kv4_read(d, 0, 2, 3, 0, None, FAKE, FAKE, FAKE, FAKE, None, 256, None, 256,
                                    err, None)
        return lib.ffd_kv4_write(d, 0, 2, 3, 0, None, 256, None, 256, None, FAKE, FAKE, FAKE, FAKE, err,
                                 None)
    assert call(None) == 0 and call(FAKE + 4) == 0
    assert call(FAKE + 1) == 1 and call(FAKE + 2) == 1
    bt, pos = OnGpu(torch.zeros((2, 3), dtype=torch.int32)), OnGpu(torch.zeros(2, dtype=torch.int32))
    x = OnGpu(torch.zeros((2, 2, 128), dtype=torch.bfloat16))
    cache = tuple(OnGpu(torch.zeros((4, 2, 5120), dtype=torch.uint8)) for _ in range(2))
    for bad in (torch.zeros(3, dtype=torch.uint8), torch.zeros(1, dtype=torch.float16),
                torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(ffd.FFDError) as e:
            if read:
                ffd.ffd_kv4_read(cache, pos, bt, x, x, error_word=OnGpu(bad))
            else:
                ffd.ffd_kv4_write(x, x, pos, bt, cache, error_word=OnGpu(bad))
        assert "error word" in str(e.value)


def test_import_without_a_cuda_build():
    """The package is imported where PyTorch has no CUDA, for its constants and parameters."""
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda_')]:\n"
            "    delattr(torch._C, name)\n"
            "import sparse_quantized_attention_gb300 as ffd\n"
            "assert ffd.make_kv4_params(1, 8, 2, 4, 2).max_q_len == 1\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.gpu
def test_a_step_without_tokens():
    Hkv, B = 2, 3
    cache = ffd.alloc_kv4_cache(4, Hkv)
    for t in cache:
        t.fill_(9)
    bt = torch.zeros((B, 2), dtype=torch.int32, device="cuda")
    first = torch.zeros(B, dtype=torch.int32, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    x = torch.randn((5, Hkv, 128), device="cuda").bfloat16()
    for none in (torch.empty((0, Hkv, 128), dtype=torch.bfloat16, device="cuda"), x[5:]):
        for c in (cu, None):
            ffd.ffd_kv4_write(none, none, first, bt, cache, cu_tokens=c)
            ffd.ffd_kv4_read(cache, first, bt, none, none, cu_tokens=c)
            ffd.ffd_kv4_read(cache, first, bt, none, None, cu_tokens=c)
    torch.cuda.synchronize()
    assert all(bool((t == 9).all()) for t in cache)
