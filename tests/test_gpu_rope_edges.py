"""Rotating and appending on the GPU: rows that lie between each other's."""
import pytest
import torch

import sparse_quantized_attention_gb300 as ffd
from tests.test_gpu_rope import frequencies, i32, offsets, table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [[1], [1] * 5, [33, 7], [700]])
def test_rows_of_one_wide_buffer(rows):
    """q in place inside a fused projection's rows, and q_out beside q, k and v in them: as with tensors apart."""
    gen = torch.Generator().manual_seed(5)
    Hq, Hkv, T = 20, 4, sum(rows)
    first = [10 * b for b in range(len(rows))]
    bt, P = table(first, rows, gen)
    wide = torch.randn((T, (2 * Hq + 2 * Hkv) * 128), generator=gen).to(torch.bfloat16).cuda()

    def parts(x):
        return [x[:, a * 128:b * 128].unflatten(1, (b - a, 128)) for a, b in (
            (0, Hq), (Hq, 2 * Hq), (2 * Hq, 2 * Hq + Hkv), (2 * Hq + Hkv, 2 * Hq + 2 * Hkv))]

    def call(q, out, kn, vn):
        k = torch.zeros((P, Hkv, 64, 128), dtype=torch.bfloat16, device="cuda")
        v, err = torch.zeros_like(k), i32([0])
        ffd.ffd_rope_append(q, kn, vn, frequencies(128).cuda(), i32(first), bt.cuda(), out, k, v,
                            cu_tokens=i32(offsets(rows)), error_word=err)
        assert ffd.ffd_get_error(err) == 0
        return out.clone(), k, v

    want = call(*[x.contiguous() for x in parts(wide)])
    x = wide.clone()
    q, out, kn, vn = parts(x)
    got = call(q, out, kn, vn)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(x[:, :Hq * 128], wide[:, :Hq * 128]) and torch.equal(x[:, 2 * Hq * 128:], wide[:, 2 * Hq * 128:])
    x = wide.clone()
    q, _, kn, vn = parts(x)
    got = call(q, q, kn, vn)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(x[:, Hq * 128:], wide[:, Hq * 128:])
    # over k_new's rows, v_new's, and the cache's
    x = wide.clone()
    q, _, kn, vn = parts(x)
    k = torch.zeros((max(P, T), Hkv, 64, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    small = q[:, :Hkv]
    for out in (kn, vn, k.view(-1, Hkv, 128)[:T], v.view(-1, Hkv, 128)[-T:]):
        with pytest.raises(ffd.FFDError):
            ffd.ffd_rope_append(small, kn, vn, None, i32(first), bt.cuda(), out, k, v, cu_tokens=i32(offsets(rows)))
    with pytest.raises(ffd.FFDError):
        ffd.ffd_rope_append(None, kn, vn, None, i32(first), bt.cuda(), None, k, k, cu_tokens=i32(offsets(rows)))
    torch.cuda.synchronize()
    assert torch.equal(x, wide) and not bool(k.any()) and not bool(v.any())
