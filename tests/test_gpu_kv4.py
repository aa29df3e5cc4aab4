"""The 4-bit cache on the GPU against the 64-bit statements of tests/kv4_refs.py: records byte for
byte, values exactly, attention within the bounds that kv4_refs.tolerance derives."""
import math

import pytest
import torch

import sparse_quantized_attention_gb300 as ffd
from tests import kv4_refs as R

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def offsets(counts):
    c = [0]
    for n in counts:
        c.append(c[-1] + n)
    return c


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def table(lens, gen, spare=0, width=None):
    """Random page order; the block table's unused entries are out of range."""
    nb = [(n + 63) // 64 for n in lens]
    P = max(1, sum(nb) + spare)
    perm = torch.randperm(P, generator=gen)
    bt = torch.full((len(lens), width or max(1, max(nb))), 1 << 30, dtype=torch.int32)
    at = 0
    for b, n in enumerate(nb):
        bt[b, :n] = perm[at:at + n].to(torch.int32)
        at += n
    return bt, P


# ---- write and read -----------------------------------------------------------------------------
ROW_CASES = [
    # (KV heads, first token of each sequence, rows of each sequence)
    ("one_token", 2, [0], [1]),
    ("step", 8, [5, 63, 64, 127, 200, 1, 0], [1, 1, 1, 1, 1, 1, 1]),
    ("ragged", 4, [0, 61, 30], [65, 7, 129]),
    ("some_empty", 1, [3, 0, 9], [0, 70, 0]),
    ("three_heads", 3, [17], [200]),
]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("name,Hkv,first,rows", ROW_CASES, ids=[c[0] for c in ROW_CASES])
def test_write_then_read(name, Hkv, first, rows, dtype):
    gen = torch.Generator().manual_seed(len(name) * 7 + Hkv)
    bt, P = table([f + r for f, r in zip(first, rows)], gen, spare=2)
    cu = offsets(rows)
    lead, T = 3, cu[-1]  # rows before the first sequence and behind the last one belong to nobody
    wide = torch.randn((T + 2 * lead, 2 * Hkv * 128 + 8), generator=gen).to(dtype)
    kx, vx = wide[:, :Hkv * 128], wide[:, Hkv * 128 + 8:]
    dev = wide.cuda()
    k_new = dev[:, :Hkv * 128].unflatten(1, (Hkv, 128))
    v_new = dev[:, Hkv * 128 + 8:].unflatten(1, (Hkv, 128))
    before = torch.randint(0, 256, (2, P, Hkv, 5120), generator=gen, dtype=torch.int32)
    before = before.to(torch.uint8)
    cache = ffd.Kv4Cache(before[0].cuda(), before[1].cuda())
    cu_dev = i32([lead + c for c in cu])
    err = i32([0])
    ffd.ffd_kv4_write(k_new, v_new, i32(first), bt.cuda(), cache, cu_tokens=cu_dev, error_word=err)
    assert ffd.ffd_get_error(err) == 0
    page, row, head, src = [], [], [], []
    for b, r in enumerate(rows):
        for i in range(r):
            p = first[b] + i
            for h in range(Hkv):
                page.append(int(bt[b, p // 64]))
                row.append(p % 64)
                head.append(h)
                src.append((lead + cu[b] + i, h))
    for x, rec, got in ((kx, before[0].clone(), cache.k4), (vx, before[1].clone(), cache.v4)):
        R.put_rows(rec, page, row, head,
                   torch.stack([x[t].reshape(Hkv, 128)[h] for t, h in src]))
        assert torch.equal(got.cpu(), rec)
    # read back into rows of their own width, in both types
    for out_type in (BF16, F16):
        back = torch.full((T + 2 * lead, 2 * Hkv * 128 + 16), 7.0, dtype=out_type, device="cuda")
        ko = back[:, :Hkv * 128].unflatten(1, (Hkv, 128))
        vo = back[:, Hkv * 128 + 16:].unflatten(1, (Hkv, 128))
        ffd.ffd_kv4_read(cache, i32(first), bt.cuda(), ko, vo, cu_tokens=cu_dev, error_word=err)
        assert ffd.ffd_get_error(err) == 0
        want = torch.full_like(back.cpu(), 7.0)
        held = R.held64(wide[lead:lead + T, :Hkv * 128].reshape(T, Hkv, 128))
        want[lead:lead + T, :Hkv * 128] = held.reshape(T, -1).half().to(out_type)
        held = R.held64(wide[lead:lead + T, Hkv * 128 + 8:].reshape(T, Hkv, 128))
        want[lead:lead + T, Hkv * 128 + 16:] = held.reshape(T, -1).half().to(out_type)
        assert torch.equal(back.cpu(), want)


def test_uniform_rows_and_one_tensor_reads():
    gen = torch.Generator().manual_seed(1)
    B, per, Hkv = 3, 5, 2
    first = [60, 0, 128]
    bt, P = table([f + per for f in first], gen)
    x = torch.randn((2, B * per, Hkv, 128), generator=gen).to(BF16)
    cache = ffd.alloc_kv4_cache(P, Hkv)
    ffd.ffd_kv4_write(x[0].cuda(), x[1].cuda(), i32(first), bt.cuda(), cache)
    for which in range(2):
        out = torch.empty((B * per, Hkv, 128), dtype=F16, device="cuda")
        ffd.ffd_kv4_read(cache, i32(first), bt.cuda(), None if which else out,
                         out if which else None)
        assert torch.equal(out.cpu().double(), R.held64(x[which]))


@pytest.mark.parametrize("kind", ["constant", "zeros", "ties", "large", "tiny", "offset", "two"])
def test_special_groups(kind):
    gen = torch.Generator().manual_seed(2)
    T = 200
    x = torch.randn((T, 1, 128), generator=gen)
    if kind == "constant":
        x = x[..., :1].expand(T, 1, 128).clone()
    elif kind == "zeros":
        x = torch.zeros_like(x)
    elif kind == "ties":  # every half level of scales that are powers of two
        x = torch.randint(0, 31, (T, 1, 128), generator=gen) * 0.5
        x[..., 0::32], x[..., 1::32] = 0.0, 15.0
        x = x * 2.0 ** torch.randint(-6, 7, (T, 1, 1), generator=gen)
    elif kind == "large":
        x = x.clamp(-4, 4) * 4096
    elif kind == "tiny":
        x = x * 2.0 ** torch.randint(-24, -8, (T, 1, 1), generator=gen)
    elif kind == "offset":
        x = x * 0.01 + 100
    elif kind == "two":
        x = torch.where(x > 0, 3.0, -1.0)
    for dtype in (BF16, F16):
        y = x.to(dtype)
        bt, P = table([T], gen)
        cache = ffd.alloc_kv4_cache(P, 1)
        err = i32([0])
        ffd.ffd_kv4_write(y.cuda(), y.cuda(), i32([0]), bt.cuda(), cache, error_word=err)
        assert ffd.ffd_get_error(err) == 0
        out = torch.empty((T, 1, 128), dtype=F16, device="cuda")
        ffd.ffd_kv4_read(cache, i32([0]), bt.cuda(), out, None)
        assert torch.equal(out.cpu().double(), R.held64(y)), kind


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
def test_values_next_to_a_boundary(dtype):
    """Values a step of the type below, at and above every boundary between two codes, for many
    scales that are no powers of two."""
    gen = torch.Generator().manual_seed(8)
    T, Hkv = 500, 3
    lo = torch.randn((T, Hkv, 4, 1), generator=gen)
    hi = lo + 2.0 ** (6 * torch.rand((T, Hkv, 4, 1), generator=gen) - 4)
    lo, hi = lo.to(dtype), hi.to(dtype)
    scale = ((hi.float() - lo.float()) / 15).half().double()
    off = (lo.double() - 16 * scale).half().double()
    x = off + (16.5 + torch.randint(0, 15, (T, Hkv, 4, 32), generator=gen)) * scale
    x = x.to(dtype)
    bits = x.view(torch.int16) + torch.randint(-1, 2, x.shape, generator=gen).to(torch.int16)
    x = torch.where(x.float().abs() > 1e-3, bits.view(dtype), x)
    x = torch.maximum(torch.minimum(x, hi), lo)
    x[..., 5:6], x[..., 20:21] = lo, hi
    x = x.reshape(T, Hkv, 128)
    bt, P = table([T], gen)
    cache = ffd.alloc_kv4_cache(P, Hkv)
    ffd.ffd_kv4_write(x.cuda(), x.cuda(), i32([0]), bt.cuda(), cache)
    out = torch.empty((2, T, Hkv, 128), dtype=F16, device="cuda")
    ffd.ffd_kv4_read(cache, i32([0]), bt.cuda(), out[0], out[1])
    want = R.held64(x)
    assert torch.equal(out[0].cpu().double(), want) and torch.equal(out[1].cpu().double(), want)


@pytest.mark.parametrize("shift", [0, 8])
def test_rows_at_any_alignment(shift):
    """Rows 16 or 32 bytes aligned, of both widths, give the same records and values."""
    gen = torch.Generator().manual_seed(9)
    T, Hkv = 130, 2
    x = torch.randn((T, Hkv, 128), generator=gen).to(BF16)
    bt, P = table([T], gen)
    for pad in (0, 8, 16):
        wide = torch.zeros((T, Hkv * 128 + pad + shift), dtype=BF16, device="cuda")
        rows = wide[:, shift:shift + Hkv * 128].unflatten(1, (Hkv, 128))
        rows.copy_(x)
        cache = ffd.alloc_kv4_cache(P, Hkv)
        ffd.ffd_kv4_write(rows, rows, i32([0]), bt.cuda(), cache)
        back = torch.full_like(wide, 7.0)
        out = back[:, shift:shift + Hkv * 128].unflatten(1, (Hkv, 128))
        ffd.ffd_kv4_read(cache, i32([0]), bt.cuda(), None, out)
        assert torch.equal(out.cpu().double(), R.held64(x).half().to(BF16).double())
        assert bool((back[:, :shift] == 7).all()) and bool((back[:, shift + Hkv * 128:] == 7).all())


def test_write_and_read_skip_and_report():
    gen = torch.Generator().manual_seed(6)
    Hkv, B = 2, 3
    bt, P = table([64, 128, 64], gen, width=2)
    bt[2, 0] = P + 5
    x = torch.randn((B * 2, Hkv, 128), generator=gen).to(BF16).cuda()
    cache = ffd.alloc_kv4_cache(P, Hkv)
    cache.k4.fill_(9)
    cache.v4.fill_(9)
    err = i32([0])

    def write(first, k=x):
        ffd.ffd_kv4_write(k, x, i32(first), bt.cuda(), cache, error_word=err)
        return ffd.ffd_get_error(err)

    def untouched():
        return bool((cache.k4 == 9).all()) and bool((cache.v4 == 9).all())

    assert write([-1, -1, -1]) == 0 and untouched()
    assert write([-1, 128, -1]) == 5 and untouched()     # behind the block table's row
    assert write([-1, 2 ** 31 - 1, -1]) == 5 and untouched()
    assert write([-1, -1, 0]) == 5 and untouched()       # a page out of range
    assert write([-1, 127, -1]) == 5 and not untouched()  # one token fits, one does not
    out = torch.full_like(x, 5.0)
    ffd.ffd_kv4_read(cache, i32([-1, 127, 0]), bt.cuda(), out, None, error_word=err)
    assert ffd.ffd_get_error(err) == 5
    assert bool((out[:2] == 5).all())                    # a negative position: left as it was
    assert torch.equal(out[2].cpu().double(),
                       R.held64(x[2].cpu()).half().to(BF16).double())
    assert bool((out[3:] == 0).all())                    # out of range: zeros
    for bad in (math.nan, math.inf, 20000.0):
        y = x.clone()
        y[0, 1, 77] = bad
        assert write([0, -1, -1], k=y) == 6


# ---- attention ----------------------------------------------------------------------------------
class Case:
    def __init__(self, lens, qlens, Hkv, G, *, dtype=BF16, window=0, keep=None, seed=0, spare=1,
                 q_scale=1.0, max_q=None, stride_pad=0, tail=0):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.qlens, self.Hkv, self.Hq = lens, qlens, Hkv, Hkv * G
        self.dtype, self.window = dtype, window
        bt, self.P = table(lens, gen, spare=spare)
        dev = torch.Generator(device="cuda").manual_seed(seed)
        k, v = (torch.randn((self.P, Hkv, 64, 128), generator=dev, device="cuda")
                for _ in range(2))
        self.k4, self.v4 = R.pack64(k), R.pack64(v)
        self.bt = bt.cuda()
        self.cu = offsets(qlens)
        self.T = self.cu[-1] + tail
        wide = torch.randn((self.T, self.Hq * 128 + stride_pad), generator=gen) * q_scale
        self.q = wide.to(dtype).cuda()[:, :self.Hq * 128].unflatten(1, (self.Hq, 128))
        self.max_q = max_q or max(1, max(qlens))
        self.keep = None
        if keep is not None:
            self.keep = (torch.rand((len(lens), Hkv, bt.shape[1]), generator=gen) < keep)
            self.keep = self.keep.to(torch.uint8).cuda()

    def poison_unused(self):
        """NaN-making bytes in every token row at or past a sequence's length, and spare pages."""
        used = torch.zeros((self.P, 64), dtype=torch.bool)
        for b, n in enumerate(self.lens):
            for j in range((n + 63) // 64):
                used[int(self.bt[b, j]), :max(0, min(64, n - 64 * j))] = True
        for rec in (self.k4, self.v4):
            par = rec[..., 4096:].reshape(self.P, self.Hkv, 64, 16)
            par[~used.cuda()[:, None].expand(-1, self.Hkv, -1)] = 0xff

    def params(self, **kw):
        return ffd.make_kv4_params(len(self.lens), self.Hq, self.Hkv, self.P, self.bt.shape[1],
                                   max_q_len=self.max_q, total_q=self.T, dtype=self.dtype,
                                   window=self.window, q_stride=self.q.stride(0), **kw)

    def buffers(self):
        return (torch.full((self.T, self.Hq, 128), 3.0, dtype=self.dtype, device="cuda"),
                torch.full((self.T, self.Hq), 3.0, device="cuda"))

    def call(self, out, lse, ws, p, **kw):
        ffd.ffd_kv4_attention(p, self.q, ffd.Kv4Cache(self.k4, self.v4), i32(self.lens), self.bt,
                              out, ws, cu_q=i32(self.cu), keep_in=self.keep, lse=lse, **kw)

    def run(self, want_err=0, **kw):
        p = self.params(**kw)
        ws = ffd.alloc_kv4_workspace(p)
        out, lse = self.buffers()
        self.call(out, lse, ws, p)
        assert ffd.ffd_get_error(ws) == want_err
        return out, lse

    def check(self, out, lse):
        ref = R.attention64(self.q, self.k4, self.v4, self.lens, self.cu, self.bt, self.Hkv,
                            window=self.window, keep=self.keep, sm=float(self.params().sm_scale))
        tol_o, tol_l = R.tolerance(*ref, self.dtype)
        want, want_lse = ref[0], ref[1]
        mine = torch.zeros_like(want_lse, dtype=torch.bool)
        mine[self.cu[0]:self.cu[-1]] = True
        assert bool((out[~mine] == 3.0).all()) and bool((lse[~mine] == 3.0).all())
        # a query with an infinity in it leaves its own row unspecified
        mine &= torch.isfinite(self.q).all(-1)
        empty = mine & (want_lse == -math.inf)
        assert bool((out[empty] == 0).all()) and bool((lse[empty] == -math.inf).all())
        some = mine & ~empty
        d = (out.double() - want).abs()
        over = (d / tol_o)[some]
        assert bool(torch.isfinite(out[some].float()).all())
        assert over.numel() == 0 or float(over.max()) <= 1.0, f"output: {float(over.max())} of bound"
        dl = ((lse.double() - want_lse).abs() / tol_l)[some]
        assert dl.numel() == 0 or float(dl.max()) <= 1.0, f"lse: {float(dl.max())} of its bound"


DECODE = [
    ("one_token", dict(lens=[1], qlens=[1], Hkv=1, G=1)),
    ("edges", dict(lens=[0, 1, 63, 64, 65, 127, 128, 129], qlens=[1] * 8, Hkv=2, G=4)),
    ("g1", dict(lens=[300, 77], qlens=[1, 1], Hkv=3, G=1)),
    ("g2_fp16", dict(lens=[300, 77], qlens=[1, 1], Hkv=2, G=2, dtype=F16)),
    ("g3", dict(lens=[1000], qlens=[1], Hkv=1, G=3)),
    ("g5", dict(lens=[700, 64], qlens=[1, 1], Hkv=2, G=5)),
    ("g7", dict(lens=[5000, 1, 640], qlens=[1, 1, 1], Hkv=2, G=7)),
    ("g8_fp16", dict(lens=[2049], qlens=[1], Hkv=4, G=8, dtype=F16)),
    ("strided", dict(lens=[500, 900], qlens=[1, 1], Hkv=2, G=4, stride_pad=136)),
    ("peaked", dict(lens=[4096], qlens=[1], Hkv=2, G=4, q_scale=12.0)),
    ("huge_q", dict(lens=[400], qlens=[1], Hkv=1, G=4, q_scale=3e4, dtype=F16)),
    ("large_q", dict(lens=[400, 90], qlens=[1, 1], Hkv=1, G=4, q_scale=1e4, dtype=F16)),
    ("large_q_bf16", dict(lens=[400, 90], qlens=[1, 3], Hkv=1, G=4, q_scale=1e9)),
    ("tiny_q", dict(lens=[400], qlens=[1], Hkv=1, G=4, q_scale=1e-6)),
    ("window_1", dict(lens=[300, 64, 65], qlens=[1, 1, 1], Hkv=2, G=4, window=1)),
    ("window_100", dict(lens=[3000, 64, 165], qlens=[1, 1, 1], Hkv=2, G=4, window=100)),
    ("mask", dict(lens=[3000, 64, 1650], qlens=[1, 1, 1], Hkv=2, G=4, keep=0.3)),
    ("mask_none", dict(lens=[3000, 64], qlens=[1, 1], Hkv=2, G=4, keep=0.0)),
    ("no_queries", dict(lens=[300, 200, 100], qlens=[0, 1, 0], Hkv=2, G=4)),
    ("many_short", dict(lens=[1 + 7 * i % 150 for i in range(300)], qlens=[1] * 300, Hkv=2, G=4)),
    ("very_many", dict(lens=[5 * i % 97 for i in range(1100)], qlens=[i % 3 for i in range(1100)],
                       Hkv=2, G=2)),
    ("long", dict(lens=[131072 - 5], qlens=[1], Hkv=1, G=4)),
    ("windows", dict(lens=[300000, 5, 100000], qlens=[1, 1, 1], Hkv=2, G=4, splits=3)),
    ("windows_mask", dict(lens=[300000, 5, 100000], qlens=[1, 3, 2], Hkv=2, G=4, keep=0.05,
                          splits=1)),
    ("long_ragged", dict(lens=[60000, 100, 33333], qlens=[1, 1, 1], Hkv=4, G=7)),
]
SEVERAL = [
    ("two", dict(lens=[300, 65], qlens=[2, 2], Hkv=2, G=4)),
    ("verify", dict(lens=[300, 650, 64, 4], qlens=[3, 4, 1, 4], Hkv=2, G=4)),
    ("verify_g1", dict(lens=[300, 650], qlens=[16, 9], Hkv=2, G=1)),
    ("verify_g7_fp16", dict(lens=[1300, 65], qlens=[6, 5], Hkv=2, G=7, dtype=F16)),
    ("verify_25_rows", dict(lens=[1300, 65, 64], qlens=[5, 4, 1], Hkv=2, G=5)),
    ("verify_32_rows", dict(lens=[130, 6500], qlens=[4, 3], Hkv=2, G=8, window=100)),
    ("verify_33_rows", dict(lens=[130, 650], qlens=[11, 3], Hkv=2, G=3, dtype=F16)),
    ("verify_mask", dict(lens=[3000, 700], qlens=[4, 8], Hkv=2, G=4, keep=0.3)),
    ("verify_windows", dict(lens=[300000, 5, 100000], qlens=[4, 3, 2], Hkv=2, G=7, splits=2)),
    ("more_queries_than_tokens", dict(lens=[3, 0, 70], qlens=[5, 2, 80], Hkv=2, G=4)),
    ("chunk", dict(lens=[513, 200], qlens=[200, 200], Hkv=1, G=4)),
    ("chunk_g8", dict(lens=[1000], qlens=[333], Hkv=2, G=8)),
    ("chunk_g3_fp16", dict(lens=[1000, 129], qlens=[100, 129], Hkv=2, G=3, dtype=F16)),
    ("chunk_window", dict(lens=[2000, 300], qlens=[190, 300], Hkv=1, G=5, window=77)),
    ("chunk_mask", dict(lens=[2000, 300], qlens=[190, 300], Hkv=2, G=4, keep=0.4)),
    ("chunk_peaked", dict(lens=[1500], qlens=[257], Hkv=1, G=4, q_scale=10.0)),
    ("chunk_large_q", dict(lens=[500], qlens=[100], Hkv=1, G=4, q_scale=1e9)),
    ("chunk_tiny_q", dict(lens=[500], qlens=[100], Hkv=1, G=4, q_scale=1e-20)),
    ("chunk_long", dict(lens=[20000], qlens=[64], Hkv=2, G=7)),
    ("chunk_many", dict(lens=[1 + 11 * i % 170 for i in range(100)],
                        qlens=[41 * i % 50 for i in range(100)], Hkv=2, G=3)),
    ("chunk_very_many", dict(lens=[3 * i % 130 for i in range(700)],
                             qlens=[i % 40 for i in range(700)], Hkv=1, G=2)),
    ("chunk_many_long", dict(lens=[40 * i for i in range(90)], qlens=[40] * 90, Hkv=1, G=4)),
    ("chunk_prompt", dict(lens=[2500, 130], qlens=[2500, 130], Hkv=2, G=8)),
    ("chunk_prompt_window", dict(lens=[2700], qlens=[2600], Hkv=2, G=8, window=300)),
    ("tails", dict(lens=[100, 90], qlens=[20, 30], Hkv=2, G=4, tail=11, max_q=77)),
    ("mixed", dict(lens=[9000, 77, 600, 128], qlens=[1, 40, 0, 128], Hkv=2, G=6, stride_pad=8)),
]


@pytest.mark.parametrize("name,kw", DECODE + SEVERAL, ids=[c[0] for c in DECODE + SEVERAL])
def test_attention(name, kw):
    kw = dict(kw)
    splits = kw.pop("splits", 0)
    c = Case(seed=len(name) + 1, **kw)
    c.poison_unused()
    out, lse = c.run(num_splits=splits)
    c.check(out, lse)


def test_probabilities_below_the_least_step():
    """Peaked rows, one of them with a V of exactly 0 in a channel at its largest score: what is left
    there are probabilities that f16 holds with few bits or none."""
    c = Case([70, 58, 55, 9, 1, 0, 70, 0, 68, 0, 64, 70, 15, 2, 1, 52, 70, 70, 1, 70],
             [100, 0, 0, 1, 82, 1, 1, 0, 1, 7, 81, 75, 15, 1, 100, 52, 1, 0, 0, 33], 2, 6,
             window=50, seed=839755, q_scale=8.0)
    out, lse = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("q,length", [(1, 70000), (5, 70000), (70, 40000)])
def test_one_sequence_over_every_cta(q, length):
    """More CTAs share a unit than are joined at once, twice with the same workspace."""
    c = Case([length, 200], [q, 1], 1, 5, seed=17)
    p = c.params()
    ws = ffd.alloc_kv4_workspace(p)
    for _ in range(2):
        out, lse = c.buffers()
        c.call(out, lse, ws, p)
        assert ffd.ffd_get_error(ws) == 0
        c.check(out, lse)


@pytest.mark.parametrize("splits", [1, 2, 3, 17, 40, 1000])
@pytest.mark.parametrize("q", [1, 3, 7, 60])
def test_any_split_count_and_repeats(splits, q):
    c = Case([2500, 63, 700], [q, min(q, 63), q], 2, 4, seed=9)
    p = c.params(num_splits=splits)
    ws = ffd.alloc_kv4_workspace(p)
    first = None
    for _ in range(3):  # the workspace is left ready for the next call
        out, lse = c.buffers()
        c.call(out, lse, ws, p)
        assert ffd.ffd_get_error(ws) == 0
        c.check(out, lse)
        if first is not None:
            assert torch.equal(first, out)  # no order of arrival in the result
        first = out


@pytest.mark.parametrize("q", [1, 5, 100])
def test_bad_entries_are_dropped_and_reported(q):
    c = Case([700, 300], [q, q], 2, 4, seed=3)
    c.bt[0, 2] = -1
    c.bt[1, 1] = c.P
    out, lse = c.run(want_err=5)
    c.check(out, lse)


@pytest.mark.parametrize("q", [1, 5, 100])
def test_every_page_bad(q):
    c = Case([700], [q], 2, 4, seed=3)
    c.bt.fill_(-7)
    out, lse = c.run(want_err=5)
    c.check(out, lse)


def test_bad_lengths_and_offsets():
    c = Case([300, 200, 100], [2, 2, 2], 2, 4, seed=4)
    p = c.params()
    ws = ffd.alloc_kv4_workspace(p)
    good, good_lse = c.run()
    cache = ffd.Kv4Cache(c.k4, c.v4)
    for cu, kept in (([0, 2, 9, 6], [0]), ([-4, 2, 4, 6], [1, 2])):
        out, lse = c.buffers()
        ffd.ffd_kv4_attention(c.params(), c.q, cache, i32(c.lens), c.bt, out, ws, cu_q=i32(cu),
                              lse=lse)
        assert ffd.ffd_get_error(ws) == 5
        for b in kept:  # the sequences whose rows are in order are computed
            if cu[b:b + 2] == [2 * b, 2 * b + 2]:
                assert torch.equal(out[2 * b:2 * b + 2], good[2 * b:2 * b + 2])
    out, lse = c.buffers()
    ffd.ffd_kv4_attention(p, c.q, cache, i32([300, -5, 100]), c.bt, out, ws, cu_q=i32(c.cu),
                          lse=lse)
    assert ffd.ffd_get_error(ws) == 5
    assert torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:])
    assert bool((out[2:4] == 0).all()) and bool((lse[2:4] == -math.inf).all())


def test_a_nan_query_stays_in_its_row():
    c = Case([500, 300], [1, 3], 2, 4, seed=5)
    good, _ = c.run()
    c.q[0, 3, 17] = math.nan
    c.q[2, 5, 100] = math.inf
    out, _ = c.run()
    assert bool(torch.isnan(out[0, 3]).all()) and bool(torch.isnan(out[2, 5]).all())
    same = torch.ones(out.shape[:2], dtype=torch.bool)
    same[0, 3] = same[2, 5] = False
    assert torch.equal(out[same.cuda()], good[same.cuda()])


def test_uniform_queries_without_offsets():
    c = Case([500, 300], [4, 4], 2, 4, seed=5)
    good, good_lse = c.run()
    p = c.params()
    ws = ffd.alloc_kv4_workspace(p)
    out, _ = c.buffers()
    ffd.ffd_kv4_attention(p, c.q, ffd.Kv4Cache(c.k4, c.v4), i32(c.lens), c.bt, out, ws)
    assert ffd.ffd_get_error(ws) == 0
    assert torch.equal(out, good)


def test_pages_past_32_bits_of_bytes():
    """Records more than 4 GiB into the cache."""
    P, Hkv = 440_000, 2  # 4.5 GB a tensor
    cache = ffd.alloc_kv4_cache(P, Hkv)
    gen = torch.Generator().manual_seed(8)
    x = torch.randn((2, 130, Hkv, 128), generator=gen).to(BF16)
    bt = i32([[P - 1, P - 2, 423_001]])
    ffd.ffd_kv4_write(x[0].cuda(), x[1].cuda(), i32([0]), bt, cache)
    out = torch.empty((130, Hkv, 128), dtype=F16, device="cuda")
    ffd.ffd_kv4_read(cache, i32([0]), bt, None, out)
    assert torch.equal(out.cpu().double(), R.held64(x[1]))
    for nq in (1, 40):
        q = torch.randn((nq, 8, 128), generator=gen).to(BF16).cuda()
        p = ffd.make_kv4_params(1, 8, Hkv, P, 3, max_q_len=nq)
        ws = ffd.alloc_kv4_workspace(p)
        o = torch.empty_like(q)
        ffd.ffd_kv4_attention(p, q, cache, i32([130]), bt, o, ws)
        assert ffd.ffd_get_error(ws) == 0
        pages = bt[0].long()
        ref = R.attention64(q, cache.k4[pages], cache.v4[pages], [130], [0, nq],
                            i32([[0, 1, 2]]), Hkv, sm=float(p.sm_scale))
        tol, _ = R.tolerance(*ref, BF16)
        assert bool(((o.double() - ref[0]).abs() <= tol).all())


# ---- together, as a decode loop uses them -------------------------------------------------------
def test_prompt_then_captured_decode_steps():
    """A prompt's chunk is written and attended to, then single tokens: write and attention are
    captured once and replayed; every replay equals the eager calls and the 64-bit statement."""
    gen = torch.Generator().manual_seed(12)
    B, Hkv, G, steps = 3, 2, 4, 4
    prompt = [130, 61, 200]
    lens = [n + steps for n in prompt]
    bt, P = table(lens, gen)
    rows = torch.randn((2, sum(lens), Hkv, 128), generator=gen).to(BF16).cuda()
    at = offsets(lens)
    cache, twin = ffd.alloc_kv4_cache(P, Hkv), ffd.alloc_kv4_cache(P, Hkv)
    btd = bt.cuda()
    cu = i32(offsets(prompt))
    chunk = torch.cat([rows[:, at[b]:at[b] + prompt[b]] for b in range(B)], 1)
    q = torch.randn((sum(prompt), Hkv * G, 128), generator=gen).to(BF16).cuda()
    p = ffd.make_kv4_params(B, Hkv * G, Hkv, P, bt.shape[1], max_q_len=max(prompt),
                            total_q=sum(prompt))
    ws = ffd.alloc_kv4_workspace(p)
    out = torch.empty_like(q)
    for c in (cache, twin):
        ffd.ffd_kv4_write(chunk[0], chunk[1], i32([0] * B), btd, c, cu_tokens=cu)
    ffd.ffd_kv4_attention(p, q, cache, i32(prompt), btd, out, ws, cu_q=cu)
    assert ffd.ffd_get_error(ws) == 0
    ref = R.attention64(q, cache.k4, cache.v4, prompt, offsets(prompt), bt, Hkv,
                        sm=float(p.sm_scale))
    assert bool(((out.double() - ref[0]).abs() <= R.tolerance(*ref, BF16)[0]).all())
    # one token a sequence at a time
    p1 = ffd.make_kv4_params(B, Hkv * G, Hkv, P, bt.shape[1])
    k_new, v_new = (torch.empty((B, Hkv, 128), dtype=BF16, device="cuda") for _ in range(2))
    q1 = torch.empty((B, Hkv * G, 128), dtype=BF16, device="cuda")
    pos, sl = i32([0] * B), i32([1] * B)
    bufs = [(c, torch.empty_like(q1), ffd.alloc_kv4_workspace(p1)) for c in (cache, twin)]

    def step(c, o, w):
        ffd.ffd_kv4_write(k_new, v_new, pos, btd, c)
        ffd.ffd_kv4_attention(p1, q1, c, sl, btd, o, w)

    def fill(t):
        k_new.copy_(torch.stack([rows[0, at[b] + prompt[b] + t] for b in range(B)]))
        v_new.copy_(torch.stack([rows[1, at[b] + prompt[b] + t] for b in range(B)]))
        q1.copy_(torch.randn((B, Hkv * G, 128), generator=gen).to(BF16))
        pos.copy_(torch.tensor([n + t for n in prompt]))
        sl.copy_(torch.tensor([n + t + 1 for n in prompt]))

    fill(0)
    step(*bufs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*bufs[0])
    for t in range(steps):
        fill(t)
        graph.replay()
        step(*bufs[1])
        torch.cuda.synchronize()
        assert torch.equal(bufs[0][1], bufs[1][1])
        now = [n + t + 1 for n in prompt]
        ref = R.attention64(q1, cache.k4, cache.v4, now, [0, 1, 2, 3], bt, Hkv,
                            sm=float(p1.sm_scale))
        assert bool(((bufs[0][1].double() - ref[0]).abs() <= R.tolerance(*ref, BF16)[0]).all())


def test_two_captured_calls_share_a_workspace():
    c = Case([900, 400], [1, 1], 2, 4, seed=21)
    d = Case([64, 3000], [1, 1], 2, 4, seed=22)
    p, r = c.params(), d.params()
    n = max(ffd.ffd_kv4_workspace_size(p), ffd.ffd_kv4_workspace_size(r))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    outs = [c.buffers(), d.buffers()]
    graphs = []
    for case, par, (o, l) in ((c, p, outs[0]), (d, r, outs[1])):
        ints = [i32(case.lens), i32(case.cu)]
        cache = ffd.Kv4Cache(case.k4, case.v4)

        def call(case=case, par=par, o=o, l=l, ints=ints, cache=cache):
            ffd.ffd_kv4_attention(par, case.q, cache, ints[0], case.bt, o, ws, cu_q=ints[1], lse=l)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, ints, cache))
    for _ in range(3):
        for g, _, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert ffd.ffd_get_error(ws) == 0
    c.check(*outs[0])
    d.check(*outs[1])


def test_two_streams_at_once():
    cases = [Case([20000, 400], [1, 2], 2, 4, seed=31), Case([64, 9000], [50, 1], 2, 4, seed=32)]
    streams = [torch.cuda.Stream() for _ in cases]
    held = []
    for c in cases:
        p = c.params()
        held.append((p, ffd.alloc_kv4_workspace(p), c.buffers(), i32(c.lens), i32(c.cu)))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, (p, ws, (o, l), sl, cu) in zip(cases, streams, held):
            ffd.ffd_kv4_attention(p, c.q, ffd.Kv4Cache(c.k4, c.v4), sl, c.bt, o, ws, cu_q=cu, lse=l,
                                  stream=s)
    torch.cuda.synchronize()
    for c, (p, ws, (o, l), _, _) in zip(cases, held):
        assert ffd.ffd_get_error(ws) == 0
        c.check(o, l)


def test_over_a_selectors_mask():
    """The blocks that the framework's Top-k selector keeps on the thumbnails, attended to in the
    4-bit cache of the same tokens."""
    gen = torch.Generator().manual_seed(14)
    B, Hkv, G, n = 2, 2, 4, 2000
    lens = [n, 777]
    bt, P = table(lens, gen)
    bt = torch.where(bt < P, bt, torch.zeros_like(bt)).cuda()
    k, v = (torch.randn((P, Hkv, 64, 128), generator=gen).to(BF16).cuda() for _ in range(2))
    qc = ffd.alloc_quantized_cache(P, Hkv)
    ffd.ffd_quantize_keys(k, qc)
    cache = ffd.alloc_kv4_cache(P, Hkv)
    first, cu = i32([0] * B), i32(offsets(lens))
    rows = [torch.cat([x[bt[b].long()].transpose(1, 2).reshape(-1, Hkv, 128)[:lens[b]]
                       for b in range(B)]) for x in (k, v)]
    ffd.ffd_kv4_write(rows[0], rows[1], first, bt, cache, cu_tokens=cu)
    q = torch.randn((B, Hkv * G, 128), generator=gen).to(BF16).cuda()
    dp = ffd.make_params(B, Hkv * G, Hkv, P, bt.shape[1], sink=16, local=100)
    mask = torch.zeros((B, Hkv, bt.shape[1]), dtype=torch.uint8, device="cuda")
    ffd.ffd_select_blocks(dp, ffd.SELECT_TOPK, 5.0, q, qc, i32(lens), bt, mask,
                          ffd.alloc_select_workspace(dp))
    p = ffd.make_kv4_params(B, Hkv * G, Hkv, P, bt.shape[1])
    ws = ffd.alloc_kv4_workspace(p)
    out = torch.empty_like(q)
    ffd.ffd_kv4_attention(p, q, cache, i32(lens), bt, out, ws, keep_in=mask)
    assert ffd.ffd_get_error(ws) == 0
    ref = R.attention64(q, cache.k4, cache.v4, lens, [0, 1, 2], bt.cpu(), Hkv, keep=mask,
                        sm=float(p.sm_scale))
    assert bool(((out.double() - ref[0]).abs() <= R.tolerance(*ref, BF16)[0]).all())
