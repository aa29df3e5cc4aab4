"""What the 4-bit cache's binding and entries take and refuse besides shapes (no GPU needed)."""
import pytest
import torch

import sparse_quantized_attention_gb300 as ffd
from tests.test_kv4_host import lib, rows_call  # noqa: F401  (lib is a fixture)


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
