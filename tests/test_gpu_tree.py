"""Attention of trees of drafted tokens on the GPU against the 64-bit statement of tests/tree_refs.py,
within the bounds that it derives."""
import math

import pytest
import torch

import sparse_quantized_attention_gb300 as ffd
from tests import tree_refs as R
from tests.test_gpu_rope import i32, offsets

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


class Problem:
    """A batch over a cache of random pages; rows before the first sequence and behind the last one
    belong to nobody."""

    def __init__(self, Hq, Hkv, lens, nqs, dtype, kind="random", seed=0, lead=0, gain=1.0, spare=1,
                 width=None, wide=8):
        gen = torch.Generator().manual_seed(seed)
        self.Hq, self.Hkv, self.lens, self.nqs, self.dtype = Hq, Hkv, lens, nqs, dtype
        nb = [(n + 63) // 64 for n in lens]
        self.P = sum(nb) + spare
        perm = torch.randperm(self.P, generator=gen)
        self.bt = torch.full((len(lens), width or max(1, max(nb))), 1 << 30, dtype=torch.int32)
        at = 0
        for b, n in enumerate(nb):
            self.bt[b, :n] = perm[at:at + n].to(torch.int32)
            at += n
        self.cu = offsets(nqs, lead)
        self.T = self.cu[-1] + lead
        self.parents = None
        if kind is not None:
            self.parents = [5] * lead
            for n in nqs:
                self.parents += R.make_parents(kind, n, gen)
            self.parents += [5] * lead
        dev = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=dev, device="cuda")
        self.k = normal(self.P, Hkv, 64, 128).to(dtype)
        self.v = normal(self.P, Hkv, 64, 128).to(dtype)
        self.rows = normal(max(1, self.T), Hq * 128 + wide).to(dtype)
        self.q = self.rows[:, :Hq * 128].unflatten(1, (Hq, 128))
        if gain != 1.0:
            self.q.mul_(gain)
        self.ws = None

    def params(self, **kw):
        return ffd.make_tree_params(len(self.lens), self.Hq, self.Hkv, self.P, self.bt.shape[1],
                                    max_q_len=max(1, max(self.nqs)), total_q=max(1, self.T),
                                    q_stride=self.q.stride(0), dtype=self.dtype, **kw)

    def run(self, keep=None, want=0, parents="own", cu=None, lens=None, stream=None, lse=True, **kw):
        p = self.params(**kw)
        need = ffd.ffd_tree_workspace_size(p)
        if self.ws is None or self.ws.numel() < need:
            self.ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        out = torch.full((max(1, self.T), self.Hq, 128), 7.0, dtype=self.dtype, device="cuda")
        z = torch.full((max(1, self.T), self.Hq), 7.0, device="cuda")
        par = self.parents if isinstance(parents, str) else parents
        ffd.ffd_tree_attention(p, self.q, self.k, self.v, i32(lens or self.lens), self.bt.cuda(), out, self.ws,
                               parents=None if par is None else i32(par), cu_q=i32(cu or self.cu),
                               keep_in=None if keep is None else keep.cuda(), lse=z if lse else None,
                               stream=stream)
        assert ffd.ffd_get_error(self.ws, stream=stream) == want
        return out, z

    def check(self, keep=None, window=0, sm=None, lens=None, **kw):
        got, z = self.run(keep=keep, window=window, sm_scale=sm, lens=lens, **kw)
        ref = R.attention64(self.q, self.k, self.v, lens or self.lens, self.cu, self.bt, self.parents,
                            window=window, keep=keep, sm=sm)
        compare(got, z, ref, self.dtype)
        return got, z


def compare(got, z, ref, dtype, skip=None):
    out, lse = ref[0], ref[1]
    tol, ltol = R.tolerance(*ref, dtype)
    mine = ~torch.isnan(lse)                       # rows of some sequence
    if skip is not None:
        mine &= ~skip
    assert bool((got[torch.isnan(lse)] == 7.0).all()) and bool((z[torch.isnan(lse)] == 7.0).all())
    g, w, t = got.double()[mine], out[mine], tol[mine]
    assert bool(torch.isfinite(g).all())
    over = (g - w).abs() - t
    assert float(over.max()) <= 0, (float(over.max()), int((over > 0).sum()), over.shape)
    empty = lse == -math.inf
    assert torch.equal((z == -math.inf)[mine], empty[mine])
    assert bool((got[empty] == 0).all())
    some = mine & ~empty
    over = (z.double() - lse).abs()[some] - ltol[some]
    assert some.sum() == 0 or float(over.max()) <= 0, float(over.max())


CASES = [
    # name, Hq, Hkv, lengths (nodes among them), nodes, kind
    ("one", 1, 1, [1], [1], "random"),
    ("token", 8, 2, [100, 64, 65, 1], [1, 1, 1, 1], "random"),
    ("small", 8, 2, [300, 70, 12], [12, 7, 12], "random"),
    ("only_trees", 4, 1, [64, 33, 130], [64, 33, 130], "random"),
    ("straddle", 6, 2, [129, 66, 200], [20, 4, 75], "random"),
    ("star", 8, 8, [500], [64], "star"),
    ("forest", 14, 2, [129, 500], [40, 61], "forest"),
    ("binary", 16, 2, [1000], [127], "binary"),
    ("chain_nodes", 5, 1, [700], [90], "chain"),
    ("chain", 5, 1, [700, 90], [90, 90], None),
    ("most", 8, 1, [256, 900], [256, 256], "random"),
    ("g7", 7, 1, [1000, 200], [19, 18], "random"),
    ("g3", 12, 4, [400, 64], [43, 42], "random"),
    ("none_between", 8, 4, [100, 50, 0, 300], [5, 0, 0, 9], "random"),
    ("longer", 8, 2, [5000], [30], "random"),
    ("chunk", 8, 2, [600, 700], [600, 333], None),
    ("tokens_of_many", 4, 2, [64 * (b % 5) + b + 1 for b in range(70)], [1] * 70, "random"),
]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_against_64_bits(case, dtype):
    name, Hq, Hkv, lens, nqs, kind = case
    x = Problem(Hq, Hkv, lens, nqs, dtype, kind, seed=len(name), lead=2)
    x.check()
    for window in (1, 3, 70):
        x.check(window=window)


@pytest.mark.parametrize("rows", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256])
@pytest.mark.parametrize("G", [1, 2, 5, 8])
def test_numbers_of_rows(rows, G):
    """Nodes around the sizes of tiles, over a few pages with an odd and an even number of them."""
    for n in (rows + 100, rows + 200):
        Problem(G, 1, [n], [rows], F16, seed=rows).check()


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 191, 192, 193, 320, 1023, 1024, 1025])
def test_lengths(n):
    for nq in {1, min(n, 5), min(n, 64), min(n, 65)}:
        Problem(4, 2, [n, n], [nq, 1], BF16, seed=n).check()


@pytest.mark.parametrize("splits", [0, 1, 2, 3, 5, 16, 100, 1000])
def test_splits(splits):
    x = Problem(8, 2, [4000, 1, 777, 2500], [12, 1, 30, 9], F16, seed=1)
    x.check(num_splits=splits)
    x.check(num_splits=splits, window=1000)
    x = Problem(8, 1, [2000, 300], [100, 70], BF16, seed=2)  # several groups of rows
    x.check(num_splits=splits)


def test_long_sequences():
    x = Problem(7, 1, [140000, 70000], [20, 33], BF16, seed=3)
    x.check()
    x.check(window=100000)
    x = Problem(8, 1, [40000], [200], F16, seed=4)
    x.check()


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
def test_block_masks(dtype):
    x = Problem(8, 2, [1000, 300, 65, 40], [20, 64, 3, 2], dtype, seed=5, lead=1)
    gen = torch.Generator().manual_seed(5)
    shape = (4, 2, x.bt.shape[1])
    for share in (0.0, 0.1, 0.5, 0.9):
        keep = (torch.rand(shape, generator=gen) < share).to(torch.uint8) * 3
        x.check(keep=keep)
        x.check(keep=keep, window=100)
    keep = torch.zeros(shape, dtype=torch.uint8)
    keep[:, :, 0] = 1                              # most rows see the first block alone
    x.check(keep=keep)
    x.check(keep=keep, num_splits=3)


def test_dropped_blocks_need_no_pages():
    x = Problem(8, 2, [1000], [20], F16, seed=6)
    keep = torch.ones((1, 2, 16), dtype=torch.uint8)
    keep[:, :, 3:9] = 0
    x.bt[:, 3:9] = -5
    x.check(keep=keep)
    x.bt[:, 3:9] = 1 << 30
    x.check(keep=keep)


def test_rows_one_mask_after_another_leaves_empty():
    """A tree's own block dropped: with a window the nodes deep in it see nothing, the others do."""
    x = Problem(4, 1, [64 + 40], [40], F16, "chain", seed=7)
    keep = torch.tensor([[[1, 0]]], dtype=torch.uint8)
    got, z = x.check(keep=keep, window=10)
    assert bool((z[:9] > -math.inf).all()) and bool((z[9:] == -math.inf).all())


@pytest.mark.parametrize("gain", [0.0, 30.0, 1000.0, 60000.0])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
def test_peaked_scores(gain, dtype):
    x = Problem(8, 2, [3000, 100], [20, 30], dtype, seed=8, gain=gain if gain < 60000 else 15000.0)
    x.check()
    if gain:
        # scores that rise towards the end, so that references are raised again and again
        order = torch.argsort((x.q[0, 0].float() @ x.k[:, 0].float().flatten(0, 1).T))
        flat = x.k[:, 0].flatten(0, 1)[order].reshape(x.P, 64, 128)
        x.k[:, 0] = flat
        x.bt[0, :47] = torch.arange(47, dtype=torch.int32)
        x.check()


def test_scores_past_2_24():
    x = Problem(4, 1, [500], [10], F16, seed=9, gain=100.0)
    x.k.mul_(100.0)
    x.check(sm=30.0)


def test_equal_scores_and_one_value():
    x = Problem(8, 2, [1500], [40], BF16, seed=10, gain=0.0)
    x.v.fill_(3.0)
    got, z = x.check()
    assert bool((got == 3.0).all())
    mine, depth = R.related(x.parents)
    want = torch.log(1460.0 + 1 + depth.double()).cuda()
    assert float((z.double() - want[:, None]).abs().max()) < 2e-5


def poison(x, token, b=0, what=math.nan, tensors=("k", "v")):
    page, row = int(x.bt[b, token // 64]), token % 64
    for t in tensors:
        getattr(x, t)[page, :, row] = what


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
def test_unseen_tokens_may_hold_anything(what, dtype):
    # past the sequence, in its last page and in others; behind every window
    x = Problem(8, 2, [200, 70], [10, 3], dtype, seed=11, spare=3)
    used = set(x.bt[0, :4].tolist() + x.bt[1, :2].tolist())
    for p in set(range(x.P)) - used:
        x.k[p], x.v[p] = what, what
    for t in range(200, 256):
        poison(x, t, what=what)
    for t in range(70, 128):
        poison(x, t, b=1, what=what)
    x.check()
    for t in range(0, 200 - 10 - 20 + 1):
        poison(x, t, what=what)
    for t in range(0, 70 - 3 - 20 + 1):
        poison(x, t, b=1, what=what)
    x.check(window=20)


@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("tensor", ["k", "v"])
@pytest.mark.parametrize("Hq,nq", [(8, 10), (8, 40), (8, 200)])
def test_a_branch_does_not_reach_another(what, tensor, Hq, nq):
    """An infinity or a NaN in a node's key or value leaves the rows that do not see it as they are."""
    x = Problem(Hq, 1, [150 + nq], [nq], BF16, seed=12)
    clean, cz = x.check()
    bad = nq - 4
    poison(x, 150 + bad, what=what, tensors=(tensor,))
    got, z = x.run()
    mine, _ = R.related(x.parents)
    sees = mine[:, bad].cuda()
    assert torch.equal(got[~sees], clean[~sees]) and torch.equal(z[~sees], cz[~sees])
    if tensor == "v":  # p times an infinity is one, summed with others of its sign
        assert not bool(torch.isfinite(got[sees]).any())
    # a chain's: rows before it; and through a window, those that have left it behind
    x = Problem(Hq, 1, [nq + 150], [nq], F16, None, seed=13)
    clean, cz = x.check(window=5)
    poison(x, 150 + nq - 8, what=what, tensors=(tensor,))
    got, z = x.run(window=5)
    sees = torch.zeros(nq, dtype=torch.bool, device="cuda")
    sees[nq - 8:nq - 3] = True
    assert torch.equal(got[~sees], clean[~sees]) and torch.equal(z[~sees], cz[~sees])


def test_a_bad_query_keeps_to_itself():
    for what in (math.nan, math.inf):
        x = Problem(8, 2, [700], [30], BF16, seed=14)
        clean, cz = x.run()
        x.q[11, 3, 7] = what
        got, z = x.run()
        other = torch.ones((30, 8), dtype=torch.bool, device="cuda")
        other[11, 3] = False
        assert torch.equal(got[other], clean[other]) and torch.equal(z[other], cz[other])


def test_out_of_range():
    x = Problem(4, 2, [300, 200], [10, 6], F16, seed=15)
    one = dict(num_splits=1)  # bits are compared: how the batch is cut decides how sums are grouped
    good, gz = x.run(**one)
    # a page: the block is as if dropped
    old = int(x.bt[0, 2])
    for page in (-1, x.P, 1 << 30):
        x.bt[0, 2] = page
        x.check(want=5)
    x.bt[0, 2] = old
    # a parent: as -1
    bad = list(x.parents)
    for p in (7, 9, -2, 1 << 30):
        bad[7] = p
        got, z = x.run(parents=bad, want=5, **one)
        bad[7] = -1
        same, sz = x.run(parents=bad, **one)
        assert torch.equal(got, same) and torch.equal(z, sz)
    # a length below the nodes': nothing is seen; above the table's: clamped
    for n in (9, 0, -4):
        got, z = x.run(lens=[n, 200], want=5, **one)
        assert bool((got[:10] == 0).all()) and bool((z[:10] == -math.inf).all())
        assert torch.equal(got[10:], good[10:])
    got, z = x.run(lens=[64 * x.bt.shape[1] + 1, 200], want=5, **one)
    full, fz = x.run(lens=[64 * x.bt.shape[1], 200], **one)
    assert torch.equal(got, full)
    # offsets
    for cu in ([-1, 10, 16], [11, 10, 16], [0, 1 << 30, 16], [0, 11, 17]):
        got, z = x.run(cu=cu, want=5, **one)
        if cu[1] == 10:
            assert bool((got[:10] == 7).all()) and torch.equal(got[10:], good[10:])
    assert x.run(**one)[0].equal(good)


def test_strides_and_no_lse():
    for wide in (0, 8, 1000):
        x = Problem(6, 3, [222, 40], [9, 4], BF16, seed=16, wide=wide)
        got, _ = x.check()
        assert torch.equal(x.run(lse=False)[0], got)


def test_uniform_batches_without_offsets():
    x = Problem(8, 2, [222, 40, 300], [9, 9, 9], F16, seed=17)
    want, wz = x.check()
    out, lse = torch.empty_like(want), torch.empty_like(wz)
    for t, l in ((None, None), (lse, lse)):
        ffd.ffd_tree_attention(x.params(), x.q, x.k, x.v, i32(x.lens), x.bt.cuda(), out, x.ws,
                               parents=i32(x.parents), lse=t)
        assert torch.equal(out, want)
    assert torch.equal(lse, wz)


def test_the_same_bits_every_time():
    x = Problem(8, 2, [9000, 500, 3000], [25, 61, 8], BF16, seed=18)
    first = x.run()
    for _ in range(5):
        again = x.run()
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_graphs_streams_and_a_shared_workspace():
    x = Problem(8, 2, [4000, 300], [25, 61], F16, seed=19)
    y = Problem(4, 1, [9000], [3], F16, seed=20)
    z = Problem(8, 1, [1500], [120], F16, seed=21)
    want = [p.run() for p in (x, y, z)]
    size = max(p.ws.numel() for p in (x, y, z))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    outs, calls = [], []
    for p in (x, y, z):
        out, lse = torch.empty_like(want[0][0][:1]), None
        out = torch.zeros((p.T, p.Hq, 128), dtype=F16, device="cuda")
        lse = torch.zeros((p.T, p.Hq), device="cuda")
        outs.append((out, lse))
        calls.append((p.params(), p.q, p.k, p.v, i32(p.lens), p.bt.cuda(), out, ws))
    extra = [dict(parents=i32(p.parents), cu_q=i32(p.cu), lse=o[1]) for p, o in zip((x, y, z), outs)]
    torch.cuda.synchronize()
    graphs = []
    for c, e in zip(calls, extra):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ffd.ffd_tree_attention(*c, **e)
        graphs.append(g)
    for order in ((0, 1, 2), (2, 0, 1), (1, 1, 0, 2)):
        for o in outs:
            o[0].zero_(), o[1].zero_()
        for i in order:
            graphs[i].replay()
        assert ffd.ffd_get_error(ws) == 0
        for i in range(3):
            assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])
    side = torch.cuda.Stream()
    got = x.run(stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0][0])
    # two calls at once, each with a workspace of its own
    other = torch.zeros_like(ws)
    for o in outs:
        o[0].zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        ffd.ffd_tree_attention(*calls[0], **extra[0])
        ffd.ffd_tree_attention(*calls[2][:-1], other, **extra[2], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], want[0][0]) and torch.equal(outs[2][0], want[2][0])


def test_pages_past_32_bits():
    """Pages more than 2^31 elements into the cache."""
    Hkv, P = 8, 33000
    k = torch.zeros((P, Hkv, 64, 128), dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    dev = torch.Generator(device="cuda").manual_seed(1)
    pages = [P - 1, 3, P - 7]
    for p in pages:
        k[p] = torch.randn((Hkv, 64, 128), generator=dev, device="cuda").to(BF16)
        v[p] = torch.randn((Hkv, 64, 128), generator=dev, device="cuda").to(BF16)
    q = torch.randn((5, 16, 128), generator=dev, device="cuda").to(BF16)
    bt, par = torch.tensor([pages], dtype=torch.int32), [-1, 0, 1, 1, 3]
    p = ffd.make_tree_params(1, 16, Hkv, P, 3, max_q_len=5)
    out, lse = torch.full_like(q, 7.0), torch.full((5, 16), 7.0, device="cuda")
    ws = ffd.alloc_tree_workspace(p)
    ffd.ffd_tree_attention(p, q, k, v, i32([150]), bt.cuda(), out, ws, parents=i32(par), lse=lse)
    assert ffd.ffd_get_error(ws) == 0
    compare(out, lse, R.attention64(q, k, v, [150], [0, 5], bt, par), BF16)


def test_random_batches():
    gen = torch.Generator().manual_seed(99)

    def pick(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=gen))

    for seed in range(40):
        Hkv, G, B = pick(1, 4), pick(1, 8), pick(1, 9)
        most = (5, 20, 64, 256)[pick(0, 3)]
        nqs = [pick(0, most) for _ in range(B)]
        lens = [n + (pick(0, 3000) if pick(0, 3) else 0) for n in nqs]
        kind = ("random", "star", "forest", "chain", None)[pick(0, 4)]
        x = Problem(Hkv * G, Hkv, lens, nqs, BF16 if seed % 2 else F16, kind, seed=seed, lead=pick(0, 2),
                    width=max(1, (max(lens) + 63) // 64) + pick(0, 40))
        keep = None
        if pick(0, 2) == 0:
            keep = (torch.rand((B, Hkv, x.bt.shape[1]), generator=gen) < 0.6).to(torch.uint8)
        x.check(keep=keep, window=pick(1, 2000) if pick(0, 2) == 0 else 0)


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("nq", [3, 70])
def test_many_items_without_a_page(splits, nq):
    """One CTA meets items one after another whose blocks are all dropped, and others between them."""
    B = 12
    x = Problem(8, 2, [100 + 64 * (b % 3) for b in range(B)], [nq] * B, BF16, seed=22)
    keep = torch.zeros((B, 2, x.bt.shape[1]), dtype=torch.uint8)
    got, z = x.check(keep=keep, num_splits=splits)
    assert bool((got == 0).all())
    keep[5, 1] = 1
    keep[11, 0, 1] = 1
    x.check(keep=keep, num_splits=splits)


@pytest.mark.parametrize("splits", [0, 7, 152])
def test_sparse_masks_over_long_sequences(splits):
    """Few blocks kept of many, crowded and scattered, rows of the mask on any byte."""
    gen = torch.Generator().manual_seed(23)
    x = Problem(7, 1, [90001, 140000, 500], [25, 18, 5], BF16, seed=24, width=2201)
    keep = torch.zeros((3, 1, 2201), dtype=torch.uint8)
    keep[0, 0, 1380:1407] = 255                       # the newest, the tree's among them
    keep[0, 0, 0] = 1
    keep[1, 0, torch.randperm(2188, generator=gen)[:60]] = 128
    keep[2, 0, 7] = 2
    x.check(keep=keep, num_splits=splits)
    shifted = torch.zeros(3 * 2201 + 5, dtype=torch.uint8, device="cuda")
    shifted[5:] = keep.flatten().cuda()

    class At:                                          # a mask that begins on an odd byte
        def cuda(self):
            return shifted[5:].view(3, 1, 2201)
    got, z = x.run(keep=At(), num_splits=splits)
    want, wz = x.run(keep=keep, num_splits=splits)
    assert torch.equal(got, want) and torch.equal(z, wz)
    x.bt[1, :1000] = -7                                # kept or not, some of them are out of range
    x.check(keep=keep, num_splits=splits, want=5)


@pytest.mark.parametrize("B,Hkv", [(33, 2), (32, 8), (40, 1), (600, 1)])
def test_many_sequences(B, Hkv):
    gen = torch.Generator().manual_seed(B)
    lens = torch.randint(9, 300, (B,), generator=gen).tolist()
    nqs = torch.randint(0, 10, (B,), generator=gen).tolist()
    lens[3], nqs[3] = 5, 5
    x = Problem(2 * Hkv, Hkv, lens, nqs, F16, seed=B, lead=1)
    x.check()
    x.check(num_splits=5, window=40)
    keep = (torch.rand((B, Hkv, x.bt.shape[1]), generator=gen) < 0.5).to(torch.uint8)
    x.check(keep=keep)
    x.check(keep=keep, num_splits=3)
    # lengths that are shorter than the nodes: those rows see nothing
    lens = list(x.lens)
    for b in (1, B // 2, B - 1):
        lens[b] = max(0, nqs[b] - 1)
    x.check(lens=lens, want=5)


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("nq,lens", [(1, [100, 300]), (20, [9000, 100, 2500]), (100, [9000, 100, 2500]),
                                     (200, [200, 260])])
def test_a_wait_that_runs_out(nq, lens, splits):
    """The shortest limit, below the time of a copy: the call ends, waits for its copies before it leaves, and
    reports it or is right; on a workspace filled with zeros again the next call gives what it gave before."""
    x = Problem(8, 2, lens, [nq] * len(lens), BF16, seed=nq)
    want = x.run(num_splits=splits)
    p = x.params(num_splits=splits, wait_limit_us=1)
    args = (x.q, x.k, x.v, i32(x.lens), x.bt.cuda())
    par, cu = i32(x.parents), i32(x.cu)
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(20):
        out, z = torch.empty_like(want[0]), torch.empty_like(want[1])
        e0.record()
        ffd.ffd_tree_attention(p, *args, out, x.ws, parents=par, cu_q=cu, lse=z)
        e1.record()
        status = ffd.ffd_get_error(x.ws)
        assert e0.elapsed_time(e1) < 1500.0  # ms: no wait for what never comes (2 s)
        assert status in (0, 7)
        if status == 0:
            assert torch.equal(out, want[0]) and torch.equal(z, want[1])
        else:
            x.ws.zero_()
        again = x.run(num_splits=splits)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("splits", [0, 4, 8, 20])
def test_groups_of_a_chunk_behind_a_window(splits):
    """A chunk's groups of rows see different numbers of pages, the last not always the most."""
    for nq, n in ((90, 700), (200, 260), (120, 4000)):
        x = Problem(5, 1, [n], [nq], F16, kind=None, seed=nq)
        for window in (1, 15, 40, 64, 70, 100, 128, 150, 700):
            x.check(window=window, num_splits=splits)


@pytest.mark.parametrize("share", [0.02, 0.1, 0.5, 0.95])
@pytest.mark.parametrize("splits", [0, 1, 5])
def test_masks_of_any_density(share, splits):
    """Kept blocks are listed 512 blocks at a time and read 32 at a time: few, several batches and nearly all of
    a list, over tables whose rows begin at any byte."""
    gen = torch.Generator().manual_seed(7)
    x = Problem(8, 2, [40000, 33000, 70, 64 * 512], [8, 5, 3, 8], BF16, seed=31, width=641)
    keep = (torch.rand((4, 2, x.bt.shape[1]), generator=gen) < share).to(torch.uint8) * 0x81
    x.check(keep=keep, num_splits=splits)
    x.check(keep=keep, num_splits=splits, window=20000)


@pytest.mark.parametrize("nq", [3, 200])
def test_a_table_that_names_one_page_again_and_again(nq):
    """2^24 tokens and more, of which all blocks but the last few are one page: as that page's tokens once, each
    with the weight of its blocks. What 64 bits say of the short sequence, with the sums' rounding over up to
    1800 pages a CTA (2^-24 of l and of o each: 2.2e-4 together) on top."""
    G, tail = 4, 5
    times = 1 << 18
    n = 64 * (times + tail)
    x = Problem(G, 1, [64 * (1 + tail)], [nq], BF16, seed=nq)
    short = x.bt.clone()
    x.bt = torch.cat([short[:, :1].repeat(1, times), short[:, 1:]], dim=1)
    got, z = x.run(lens=[n])
    # by hand: scores of the short sequence, the first page's with log(times) more
    page = short[0].long().cuda()
    k = x.k[page, 0].reshape(-1, 128).double()
    v = x.v[page, 0].reshape(-1, 128).double()
    s = torch.einsum("ihd,td->iht", x.q[:nq].double(), k) / math.sqrt(128)
    s[:, :, :64] += math.log(times)
    see = torch.zeros((nq, k.shape[0]), dtype=torch.bool, device="cuda")
    see[:, :k.shape[0] - nq] = True
    for i in range(nq):
        j = i
        while j >= 0:
            see[i, k.shape[0] - nq + j] = True
            j = x.parents[j]
    s = s.masked_fill(~see[:, None, :], -math.inf)
    lse = s.logsumexp(-1)
    p = (s - lse[..., None]).exp()
    want = torch.einsum("iht,td->ihd", p, v)
    size = torch.einsum("iht,td->ihd", p, v.abs())
    # a probability is off by half a step of bf16, the result by another; the sums as above
    tol = (2.0 ** -8 + 2.2e-4) * size + 2.0 ** -8 * want.abs() + 1e-6
    assert bool(((got.double() - want).abs() <= tol).all())
    assert float((z.double() - lse).abs().max()) <= 2.2e-4 + 1e-5
