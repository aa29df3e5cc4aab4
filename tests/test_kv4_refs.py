"""Pins of the 64-bit statements of the 4-bit cache (CPU): worked groups, the record's bytes, and
attention against the definition written out."""
import math

import torch

from tests import kv4_refs as R


def test_worked_groups():
    # levels 0, 1, ..., 15 twice: scale 1, off -16, codes the levels themselves
    x = torch.tensor([float(i % 16) for i in range(32)] * 4)
    c, s, o = R.quantise64(x)
    assert s.tolist() == [1.0] * 4 and o.tolist() == [-16.0] * 4
    assert c.tolist() == [i % 16 for i in range(32)] * 4
    assert torch.equal(R.values64(c, s, o), x.double())
    # a constant group: scale 0, code 0, the value itself
    c, s, o = R.quantise64(torch.full((128,), 2.5))
    assert s.tolist() == [0.0] * 4 and o.tolist() == [2.5] * 4 and c.sum() == 0
    # half-way values: between 2 and 3 down (18 is even), between 3 and 4 up
    x[5], x[6] = 2.5, 3.5
    c, s, o = R.quantise64(x)
    assert c[5] == 2 and c[6] == 4


def test_error_bound():
    g = torch.Generator().manual_seed(3)
    x = (torch.randn((500, 128), generator=g) * 3).to(torch.bfloat16)
    c, s, o = R.quantise64(x)
    err = (R.values64(c, s, o) - x.double()).abs().reshape(500, 4, 32)
    assert bool((err <= s[..., None] / 2 + o.abs()[..., None] * 2.0 ** -11
                 + x.double().abs().reshape(500, 4, 32) * 2.0 ** -11 + 1e-6).all())


def test_record_bytes():
    x = torch.zeros((1, 1, 64, 128))
    x[0, 0, 5] = torch.tensor([float(i % 16) for i in range(32)] * 4)
    rec = R.pack64(x)[0, 0]
    # token 5 shares line 2 with token 4; word 3 (channels 24..31, levels 8..15) is in half 0:
    # sector 2 ^ 2 = 0, bytes 12 .. 15; nibbles 8 10 12 14 9 11 13 15
    at = 2 * 128 + 0 * 32 + 12
    assert rec[at:at + 4].tolist() == [0xa8, 0xec, 0xb9, 0xfd]
    # the pairs (1, -16) of token 5: f16 0x3c00, 0xcc00
    assert rec[4096 + 80:4096 + 84].tolist() == [0x00, 0x3c, 0x00, 0xcc]
    one = torch.zeros((1, 1, 5120), dtype=torch.uint8)
    for r in range(64):
        R.put_rows(one, [0], [r], [0], x[0, :, r])
    assert torch.equal(one, R.pack64(x))


def test_unpack_inverts_pack():
    g = torch.Generator().manual_seed(4)
    x = torch.randn((3, 2, 64, 128), generator=g)
    assert torch.equal(R.unpack64(R.pack64(x)), R.held64(x))
    assert len(set(R.BYTE.reshape(-1).tolist())) == 4096


def test_attention_against_the_definition():
    g = torch.Generator().manual_seed(5)
    n, nq, Hkv, G = 70, 3, 1, 2
    k4 = R.pack64(torch.randn((2, Hkv, 64, 128), generator=g))
    v4 = R.pack64(torch.randn((2, Hkv, 64, 128), generator=g))
    q = torch.randn((nq, Hkv * G, 128), generator=g)
    bt = torch.tensor([[1, 0]], dtype=torch.int32)
    out, lse, *_ = R.attention64(q, k4, v4, [n], [0, nq], bt, Hkv, window=9)
    K = torch.cat((R.unpack64(k4[1, 0]), R.unpack64(k4[0, 0])))
    V = torch.cat((R.unpack64(v4[1, 0]), R.unpack64(v4[0, 0])))
    for i in range(nq):
        p = n - nq + i
        for h in range(G):
            w = [math.exp(float(q[i, h].double() @ K[j]) / math.sqrt(128.0))
                 for j in range(p - 8, p + 1)]
            want = sum(a * V[j] for a, j in zip(w, range(p - 8, p + 1))) / sum(w)
            assert torch.allclose(out[i, h], want, rtol=1e-12, atol=1e-12)
            assert abs(float(lse[i, h]) - math.log(sum(w))) < 1e-12
    # a row that sees nothing
    out, lse, *_ = R.attention64(q, k4, v4, [1], [0, nq], bt, Hkv)
    assert out[0].abs().sum() == 0 and lse[0].tolist() == [-math.inf] * 2
    assert torch.equal(out[2, 0], V[0])
