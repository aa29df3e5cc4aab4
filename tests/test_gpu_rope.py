"""Rotating and appending on the GPU against the 64-bit rotation of tests/tree_refs.py, within the
bounds that it derives; records against ffd_quantize_keys's, bit for bit."""
import pytest
import torch

import sparse_quantized_attention_gb300 as ffd
from tests import tree_refs as R

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(counts, lead=0):
    c = [lead]
    for n in counts:
        c.append(c[-1] + n)
    return c


def table(first, rows, gen, spare=1):
    """Block table over randomly ordered pages; entries before a sequence's first new token and behind
    its last one are out of range."""
    nb = [(f + r + 63) // 64 - f // 64 if r else 0 for f, r in zip(first, rows)]
    P = sum(nb) + spare
    perm = torch.randperm(P, generator=gen)
    bt = torch.full((len(first), max(1, max((f + r + 63) // 64 for f, r in zip(first, rows)))), 1 << 30,
                    dtype=torch.int32)
    at = 0
    for b, n in enumerate(nb):
        bt[b, first[b] // 64:first[b] // 64 + n] = perm[at:at + n].to(torch.int32)
        at += n
    return bt, P


def frequencies(rot):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (10000.0 ** (-2.0 * i / rot)).float() if rot else None


def near(got, want, err, what):
    off = (got.double() - want).abs() - err
    assert not torch.isnan(got.double()).any(), what
    assert float(off.max()) <= 0, (what, float(off.max()), int((off > 0).sum()))


CASES = [
    # name, Hq, Hkv, first token and rows of each sequence, rotated channels, interleaved, scale
    ("one", 1, 1, [0], [1], 128, False, 1.0),
    ("step", 28, 4, [131071, 5, 63, 64, 0], [1, 1, 1, 1, 1], 128, False, 1.0),
    ("ragged", 8, 2, [61, 0, 1000, 3], [65, 7, 0, 129], 128, False, 1.0),
    ("pairs", 6, 3, [100, 4095], [33, 2], 128, True, 1.0),
    ("half", 5, 5, [17], [70], 64, False, 1.0),
    ("half_pairs", 16, 2, [17, 200], [20, 3], 64, True, 0.75),
    ("some", 7, 1, [90000], [40], 96, False, 1.25),
    ("some_pairs", 8, 8, [3], [9], 96, True, 1.0),
    ("least", 4, 2, [250000], [5], 16, False, 1.0),
    ("least_pairs", 4, 2, [250000], [5], 16, True, -2.0),
    ("none", 4, 2, [9], [80], 0, False, 1.0),
    ("long", 8, 2, [1000], [9000], 128, False, 1.0),
]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_against_64_bits(case, dtype):
    name, Hq, Hkv, first, rows, rot, inter, scale = case
    gen = torch.Generator().manual_seed(len(name) + 10 * Hq)
    bt, P = table(first, rows, gen)
    lead, T = 2, sum(rows)  # rows before the first sequence and behind the last belong to nobody
    wide = torch.randn((T + 2 * lead, (Hq + 2 * Hkv) * 128 + 8), generator=gen).to(dtype).cuda()
    q = wide[:, :Hq * 128].unflatten(1, (Hq, 128))
    kn = wide[:, Hq * 128:(Hq + Hkv) * 128].unflatten(1, (Hkv, 128))
    vn = wide[:, (Hq + Hkv) * 128 + 8:].unflatten(1, (Hkv, 128))
    before = torch.randn((2, P, Hkv, 64, 128), generator=gen).to(dtype).cuda()
    k, v = before[0].clone(), before[1].clone()
    out = torch.full((T + 2 * lead, Hq + 1, 128), 7.0, dtype=dtype, device="cuda")[:, :Hq]
    freq = frequencies(rot)
    err = i32([0])
    args = dict(cu_tokens=i32(offsets(rows, lead)), interleaved=inter, rot_scale=scale, error_word=err)
    ffd.ffd_rope_append(q, kn, vn, None if freq is None else freq.cuda(), i32(first), bt.cuda(), out, k, v,
                        **args)
    assert ffd.ffd_get_error(err) == 0
    tokens = torch.tensor([f + i for f, r in zip(first, rows) for i in range(r)]).cuda()
    seq = torch.tensor([b for b, r in enumerate(rows) for _ in range(r)]).cuda()
    page, row = bt.cuda()[seq, tokens // 64].long(), tokens % 64
    want, bound = R.rotated64(q[lead:lead + T], tokens, freq, inter, scale)
    near(out[lead:lead + T], want, bound, "q")
    assert bool((out[:lead] == 7).all()) and bool((out[lead + T:] == 7).all())
    want, bound = R.rotated64(kn[lead:lead + T], tokens, freq, inter, scale)
    near(k[page, :, row], want, bound, "k")
    assert torch.equal(v[page, :, row], vn[lead:lead + T])
    # nothing else of the cache is touched
    rest = torch.ones((P, 64), dtype=torch.bool, device="cuda")
    rest[page, row] = False
    for got, old in ((k, before[0]), (v, before[1])):
        assert torch.equal(got.transpose(1, 2)[rest], old.transpose(1, 2)[rest])
    # channels that are not rotated pass bit for bit
    assert torch.equal(k[page, :, row][..., rot:], kn[lead:lead + T][..., rot:])
    # in place, without queries, and by rotary positions of their own
    k2, v2 = before[0].clone(), before[1].clone()
    again = wide.clone()
    q2 = again[:, :Hq * 128].unflatten(1, (Hq, 128))
    ffd.ffd_rope_append(q2, kn, vn, None if freq is None else freq.cuda(), i32(first), bt.cuda(), q2, k2, v2,
                        **args)
    assert torch.equal(q2[lead:lead + T], out[lead:lead + T]) and torch.equal(k2, k)
    assert torch.equal(again[:, Hq * 128:], wide[:, Hq * 128:]) and torch.equal(again[:lead], wide[:lead])
    places = torch.cat([torch.zeros(lead, dtype=torch.long).cuda(), tokens,
                        torch.zeros(lead, dtype=torch.long).cuda()]).int()
    k2, v2 = before[0].clone(), before[1].clone()
    ffd.ffd_rope_append(None, kn, vn, None if freq is None else freq.cuda(), i32(first), bt.cuda(), None, k2,
                        v2, rope_positions=places, **args)
    assert torch.equal(k2, k) and torch.equal(v2, v)


def test_far_positions_and_high_frequencies():
    """Angles of up to 2^24 positions: the bound of ffd.h, 1e-6 of a turn and less, holds."""
    gen = torch.Generator().manual_seed(3)
    T = 4096
    places = torch.randint(0, 1 << 24, (T,), generator=gen)
    places[:4] = torch.tensor([0, 1, (1 << 24) - 1, 1 << 23])
    freq = torch.rand(64, generator=gen)
    freq[0], freq[1] = 1.0, 2.0 ** -20
    x = torch.zeros((T, 1, 128), dtype=F16)
    x[..., :64] = 1.0
    bt, P = table([0], [T], gen)
    k = torch.zeros((P, 1, 64, 128), dtype=F16, device="cuda")
    v = torch.zeros_like(k)
    err = i32([0])
    ffd.ffd_rope_append(None, x.cuda(), x.cuda(), freq.cuda(), i32([0]), bt.cuda(), None, k, v,
                        rope_positions=places.int().cuda(), error_word=err)
    assert ffd.ffd_get_error(err) == 0
    t = torch.arange(T)
    got = k[bt[0, t // 64].long().cuda(), :, (t % 64).cuda()].double().cpu()[:, 0]
    angle = places.double()[:, None] * freq.double()
    want = torch.cat((angle.cos(), angle.sin()), -1)
    # 2^24 radians are 2^21.4 turns: two-part products of 2^-48 leave 2^-26, and 2^-25.4 as below
    bound = 2 ** -11 * want.abs() + 2 * 3.1416 * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -25
    assert bool(((got - want).abs() <= bound).all())


def test_out_of_range():
    Hq, Hkv, T = 2, 2, 5
    x = torch.randn((T, 2, 128), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    f = frequencies(128).cuda()
    bt = i32([[0, 1], [2, 77]])
    k = torch.zeros((3, Hkv, 64, 128), dtype=BF16, device="cuda")
    v, out, err = torch.zeros_like(k), torch.full_like(x, 7.0), i32([0])

    def call(first, cu, **kw):
        k.zero_(), v.zero_(), out.fill_(7.0)
        ffd.ffd_rope_append(x, x, x, f, i32(first), bt, out, k, v, cu_tokens=i32(cu), error_word=err, **kw)
        return ffd.ffd_get_error(err)

    assert call([0, 0], [0, 3, 5]) == 0
    base = out.clone()
    # a page out of range, a token past the table: not appended, the queries are rotated all the same
    assert call([0, 62], [0, 3, 5]) == 0
    assert call([0, 63], [0, 3, 5]) == 5
    assert bool((v[2, :, 63] != 0).any()) and not bool((v[2, :, :63] != 0).any())
    assert call([127, 0], [0, 3, 5]) == 5
    assert bool((out != 7.0).any(-1).all())
    # a negative first token: nothing for that sequence
    assert call([-1, 0], [0, 3, 5]) == 0
    assert bool((out[:3] == 7.0).all()) and torch.equal(out[3:], base[3:])
    assert not bool((v[:2] != 0).any())
    # rotary positions out of range
    assert call([0, 0], [0, 3, 5], rope_positions=i32([0, 1, 2, -1, 0])) == 6
    assert torch.equal(out[:3], base[:3])
    assert call([0, 0], [0, 3, 5], rope_positions=i32([0, 1, 2, 0, 1 << 24])) == 6
    assert call([0, 0], [0, 3, 5], rope_positions=i32([0, 1, 2, 0, (1 << 24) - 1])) == 0
    # offsets that skip rows or go past them
    assert call([0, 0], [1, 1, 4]) == 0
    assert bool((out[0] == 7.0).all()) and bool((out[4] == 7.0).all())
    assert call([0, 0], [0, 2, 1 << 30]) == 0


def test_infinities_and_nan_stay_where_they_are():
    x = torch.randn((2, 1, 128), generator=torch.Generator().manual_seed(1)).to(F16)
    x[0, 0, 5], x[1, 0, 100] = float("inf"), float("nan")
    k = torch.zeros((1, 1, 64, 128), dtype=F16, device="cuda")
    v = torch.zeros_like(k)
    ffd.ffd_rope_append(None, x.cuda(), x.cuda(), frequencies(64).cuda(), i32([3]), i32([[0]]), None, k, v)
    bad = ~torch.isfinite(k[0, 0, 3:5].cpu())
    assert bad[0].nonzero().flatten().tolist() == [5, 37]  # the pair's two channels
    assert bad[1].nonzero().flatten().tolist() == [100]    # not rotated: as it was
    assert torch.equal(v[0, 0, 3:5].cpu().view(torch.int16), x[:, 0].view(torch.int16))


@pytest.mark.parametrize("rows,first,rot,inter,Hkv", [
    ([1] * 9, [0, 63, 64, 100, 5000, 1, 2, 3, 4], 128, False, 4), ([300], [77], 128, True, 2),
    ([65, 1, 0, 7], [3, 0, 5, 190], 64, False, 3)])
@pytest.mark.parametrize("keep_raw", [True, False])
def test_records(rows, first, rot, inter, Hkv, keep_raw):
    """Records hold what the whole-page quantiser writes for the rotated keys."""
    gen = torch.Generator().manual_seed(sum(rows))
    bt, P = table(first, rows, gen)
    T, Hq = sum(rows), 3
    x = torch.randn((T, Hq + 2 * Hkv, 128), generator=gen).to(BF16).cuda()
    q, kn, vn = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    k = torch.randn((P, Hkv, 64, 128), generator=gen).to(BF16).cuda()
    v = torch.zeros_like(k)
    cache = ffd.alloc_quantized_cache(P, Hkv)
    ffd.ffd_quantize_keys(k, cache)
    err = i32([0])
    cu = i32(offsets(rows))
    out = torch.empty((T, Hq, 128), dtype=BF16, device="cuda")
    plain = k.clone()
    call = dict(cu_tokens=cu, interleaved=inter, error_word=err)
    f = frequencies(rot).cuda()
    ffd.ffd_rope_append(q, kn, vn, f, i32(first), bt.cuda(), torch.empty_like(out), plain,
                        torch.zeros_like(v), **call)
    ffd.ffd_rope_append(q, kn, vn, f, i32(first), bt.cuda(), out, k if keep_raw else None, v,
                        quantized=cache, **call)
    assert ffd.ffd_get_error(err) == 0
    if keep_raw:
        assert torch.equal(k, plain)
    want = ffd.alloc_quantized_cache(P, Hkv)
    ffd.ffd_quantize_keys(plain, want)
    assert torch.equal(cache.thumb, want.thumb) and torch.equal(cache.resid, want.resid)
    # a key outside the fp16 range
    kn[0, 0, 3] = 1e6
    ffd.ffd_rope_append(None, kn, vn, f, i32(first), bt.cuda(), None, None, v, quantized=cache, **call)
    assert ffd.ffd_get_error(err) == 6


def test_graph_stream_and_uniform_rows():
    gen = torch.Generator().manual_seed(4)
    B, per, Hq, Hkv = 3, 5, 4, 2
    first = [60, 0, 128]
    bt, P = table(first, [per] * B, gen)
    x = torch.randn((B * per, Hq + 2 * Hkv, 128), generator=gen).to(F16).cuda()
    q, kn, vn = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    f, pos, tab = frequencies(128).cuda(), i32(first), bt.cuda()
    k1 = torch.zeros((P, Hkv, 64, 128), dtype=F16, device="cuda")
    v1, o1 = torch.zeros_like(k1), torch.empty((B * per, Hq, 128), dtype=F16, device="cuda")
    k2, v2, o2 = torch.zeros_like(k1), torch.zeros_like(k1), torch.empty_like(o1)
    ffd.ffd_rope_append(q, kn, vn, f, pos, tab, o1, k1, v1, cu_tokens=i32([0, 5, 10, 15]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ffd.ffd_rope_append(q, kn, vn, f, pos, tab, o2, k2, v2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, o2) and torch.equal(k1, k2) and torch.equal(v1, v2)
    x.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, -o2) and torch.equal(v1, -v2)
    k2.zero_(), v2.zero_(), o2.zero_()
    torch.cuda.synchronize()
    ffd.ffd_rope_append(q, kn, vn, f, pos, tab, o2, k2, v2, stream=side)
    side.synchronize()
    assert torch.equal(o1, -o2) and torch.equal(k1, -k2)


def test_no_rows():
    bt = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    none = torch.empty((0, 2, 128), dtype=BF16, device="cuda")
    k = torch.full((1, 2, 64, 128), 9.0, dtype=BF16, device="cuda")
    v = k.clone()
    ffd.ffd_rope_append(none, none, none, frequencies(128).cuda(), i32([0, 0]), bt, none, k, v)
    ffd.ffd_rope_append(None, none, none, None, i32([0, 0]), bt, None, k, v, cu_tokens=i32([0, 0, 0]))
    torch.cuda.synchronize()
    assert bool((k == 9).all()) and bool((v == 9).all())


def test_pages_past_32_bits():
    """A cache whose last pages lie more than 2^31 elements in."""
    Hkv, P = 8, 33000                      # 33000 * 8 * 64 * 128 = 2.16e9 elements
    k = torch.zeros((P, Hkv, 64, 128), dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    x = torch.randn((2, Hkv, 128), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    err = i32([0])
    ffd.ffd_rope_append(None, x, x, None, i32([63, 5]), i32([[P - 1], [P - 2]]), None, k, v, error_word=err)
    assert ffd.ffd_get_error(err) == 0
    for t, (p, r) in enumerate(((P - 1, 63), (P - 2, 5))):
        assert torch.equal(k[p, :, r], x[t]) and torch.equal(v[p, :, r], x[t])
    assert int((v[-4:] != 0).any(-1).sum()) == 2 * Hkv and not bool(v[:4].any())


def test_token_indexes_past_the_rotary_range():
    """Without positions of their own, tokens from 2^24 on are appended and reported; with them they are fine."""
    Hkv, width = 1, (1 << 18) + 1
    bt = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    bt[0, -1] = 1
    x = torch.randn((3, Hkv, 128), generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    k = torch.zeros((2, Hkv, 64, 128), dtype=BF16, device="cuda")
    v, err, f = torch.zeros_like(k), i32([0]), frequencies(128).cuda()
    first = (1 << 24) - 1
    ffd.ffd_rope_append(None, x, x, f, i32([first]), bt, None, k, v, error_word=err)
    assert ffd.ffd_get_error(err) == 6
    assert torch.equal(v[0, 0, 63], x[0, 0]) and torch.equal(v[1, 0, :2], x[1:, 0])
    kept = k[0, 0, 63].clone()
    ffd.ffd_rope_append(None, x, x, f, i32([first]), bt, None, k, v, error_word=err,
                        rope_positions=i32([first, 0, 0]))
    assert ffd.ffd_get_error(err) == 0
    assert torch.equal(k[0, 0, 63], kept) and torch.equal(k[1, 0, :2], x[1:, 0])
