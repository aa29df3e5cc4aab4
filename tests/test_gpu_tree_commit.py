"""Committing a drafted path on the GPU against a walk in Python: results and every cache row exactly."""
import pytest
import torch

import sparse_quantized_attention_gb300 as ffd
from tests import tree_refs as R
from tests.test_gpu_rope import i32, offsets, table

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def i64(x):
    return torch.tensor(x, dtype=torch.int64, device="cuda")


def tokens(parents, luck, gen):
    """Drafted tokens and targets of one tree: a node is confirmed with probability `luck`."""
    n = len(parents)
    draft = torch.randint(0, 50, (n,), generator=gen).tolist()
    target = torch.randint(50, 100, (n,), generator=gen).tolist()
    for i, p in enumerate(parents):
        if p >= 0 and float(torch.rand(1, generator=gen)) < luck:
            target[p] = draft[i]
    return draft, target


CASES = [
    # kind, KV heads, tokens before the tree, nodes, chance that a node is confirmed
    ("random", 4, [100, 0, 63, 64, 5000], [25, 12, 64, 1, 7], 0.7),
    ("chain", 2, [61, 10], [9, 200], 1.0),
    ("chain", 1, [3], [256], 0.99),
    ("star", 3, [60, 1], [16, 200], 0.5),
    ("binary", 8, [127], [255], 0.9),
    ("forest", 2, [9, 9, 9], [30, 0, 5], 0.8),
    ("random", 1, [50] * 40, [11] * 40, 0.0),
    ("random", 2, [40, 200], [256, 250], 0.95),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}{i}" for i, c in enumerate(CASES)])
@pytest.mark.parametrize("records", [False, True])
def test_against_a_walk(case, records):
    kind, Hkv, before, nodes, luck = case
    gen = torch.Generator().manual_seed(sum(nodes) + Hkv)
    dtype = BF16 if records else F16
    bt, P = table(before, nodes, gen)
    par, draft, target = [], [], []
    for n in nodes:
        p = R.make_parents(kind, n, gen)
        d, t = tokens(p, luck, gen)
        par, draft, target = par + p, draft + d, target + t
    lead, T = 2, sum(nodes)
    cu = offsets(nodes, lead)
    pad = lambda x, v: [v] * lead + x + [v] * lead  # noqa: E731
    k = torch.randn((P, Hkv, 64, 128), generator=gen).to(dtype).cuda()
    v = torch.randn((P, Hkv, 64, 128), generator=gen).to(dtype).cuda()
    cache = None
    if records:
        cache = ffd.alloc_quantized_cache(P, Hkv)
        ffd.ffd_quantize_keys(k, cache)
    path = torch.full((T + 2 * lead,), 77, dtype=torch.int32, device="cuda")
    B = len(nodes)
    acc, lens, nxt = i32([9] * B), i32([9] * B), i64([9] * B)
    want_k, want_v = k.clone(), v.clone()
    err = i32([0])
    ffd.ffd_tree_commit(i64(pad(draft, 1)), i64(pad(target, 1)), i32([b + n for b, n in zip(before, nodes)]),
                        bt.cuda(), k, v, path, acc, nxt, lens, parents=i32(pad(par, 99)), cu_nodes=i32(cu),
                        quantized=cache, error_word=err)
    assert ffd.ffd_get_error(err) == 0
    want_path = [77] * (T + 2 * lead)
    longest = 0
    for b, n in enumerate(nodes):
        at = cu[b] - lead
        way = R.accepted_path(draft[at:at + n], target[at:at + n], par[at:at + n])
        longest = max(longest, len(way))
        want_path[cu[b]:cu[b] + n] = way + [-1] * (n - len(way))
        assert int(acc[b]) == len(way) and int(lens[b]) == before[b] + len(way)
        assert int(nxt[b]) == (target[at + way[-1]] if n else -1)
        for to, node in enumerate(way):
            x, y = before[b] + node, before[b] + to
            for c in (want_k, want_v):
                c[int(bt[b, y // 64]), :, y % 64] = c[int(bt[b, x // 64]), :, x % 64].clone()
    assert path.tolist() == want_path
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    if luck > 0.9:
        assert longest > 3
    if records:
        want = ffd.alloc_quantized_cache(P, Hkv)
        ffd.ffd_quantize_keys(want_k, want)
        assert torch.equal(cache.thumb, want.thumb) and torch.equal(cache.resid, want.resid)


def test_chains_without_parents_or_offsets():
    gen = torch.Generator().manual_seed(5)
    B, n, Hkv = 3, 6, 2
    bt, P = table([62] * B, [n] * B, gen)
    k = torch.randn((P, Hkv, 64, 128), generator=gen).to(F16).cuda()
    v = k.neg()
    k0 = k.clone()
    draft, target = i64(list(range(B * n))), i64([x + 1 for x in range(B * n)])
    target[n + 2] = 0
    path, acc, lens, nxt = i32([0] * B * n), i32([0] * B), i32([0] * B), i64([0] * B)
    ffd.ffd_tree_commit(draft, target, i32([62 + n] * B), bt.cuda(), k, v, path, acc, nxt, lens)
    assert acc.tolist() == [6, 3, 6] and lens.tolist() == [68, 65, 68] and nxt.tolist() == [6, 0, 18]
    assert path.tolist() == [0, 1, 2, 3, 4, 5, 0, 1, 2, -1, -1, -1, 0, 1, 2, 3, 4, 5]
    assert torch.equal(k, k0) and torch.equal(v, -k0)


def test_out_of_range():
    gen = torch.Generator().manual_seed(6)
    Hkv, n = 2, 8
    bt, P = table([60, 0], [n, n], gen)
    bt = bt.cuda()
    par = [-1, 0, 0, 2, 2, 4, 4, 6]
    draft, target = i64(list(range(n)) * 2), i64([2, 0, 4, 0, 6, 0, 7, 50] * 2)  # 0 2 4 6 7
    k0 = torch.randn((P, Hkv, 64, 128), generator=gen).to(F16).cuda()
    err = i32([0])

    def call(lens, cu, parents=par * 2, tab=None, rows=2 * n):
        k = k0.clone()
        v = k0.clone()
        path, acc, new, nxt = i32([77] * rows), i32([9, 9]), i32([9, 9]), i64([9, 9])
        ffd.ffd_tree_commit(draft[:rows], target[:rows], i32(lens), bt if tab is None else tab, k, v, path,
                            acc, nxt, new, parents=i32(parents[:rows]), cu_nodes=i32(cu), error_word=err)
        return ffd.ffd_get_error(err), k, path.tolist(), acc.tolist(), nxt.tolist(), new.tolist()

    status, k, path, acc, nxt, new = call([68, 8], [0, 8, 16])
    assert status == 0 and acc == [5, 5] and nxt == [50, 50] and new == [65, 5]
    assert path == [0, 2, 4, 6, 7, -1, -1, -1] * 2
    good = k
    # lengths
    for bad in (7, -1, 64 * bt.shape[1] + 1):
        status, k, path, acc, nxt, new = call([bad, 8], [0, 8, 16])
        assert status == 5 and acc == [0, 5] and nxt == [-1, 50] and new == [bad, 5]
        assert path == [-1] * 8 + [0, 2, 4, 6, 7, -1, -1, -1]
        page = int(bt[0, 0])
        assert torch.equal(k[page], k0[page])
    # offsets
    for cu in ([-1, 8, 16], [9, 8, 16], [0, 1 << 30, 16]):
        status, k, path, acc, nxt, new = call([68, 8], cu)
        assert status == 5 and acc[0] == 0 and nxt[0] == -1 and new[0] == 68
    status, k, path, acc, nxt, new = call([68, 8], [0, 8, 17])
    assert status == 5 and acc == [5, 0] and path[8:] == [77] * 8
    # parents: taken as -1
    status, k, path, acc, nxt, new = call([68, 8], [0, 8, 16], parents=[-1, 0, 2, 2, 2, 4, 4, 6] + par)
    assert status == 5 and acc == [1, 5] and path[:8] == [0] + [-1] * 7 and nxt == [2, 50]
    # pages: rows from or to one that is out of range stay
    tab = bt.clone()
    tab[0, 1] = P
    status, k, path, acc, nxt, new = call([68, 8], [0, 8, 16], tab=tab)
    assert status == 5 and acc == [5, 5]
    page = int(bt[0, 0])
    assert torch.equal(k[page, :, 61], k0[page, :, 62]) and torch.equal(k[page, :, 62], k0[page, :, 62])
    other = int(bt[1, 0])
    assert torch.equal(k[other], good[other])


def test_more_than_256_nodes_of_a_sequence():
    k = torch.zeros((10, 1, 64, 128), dtype=F16, device="cuda")
    v = torch.zeros_like(k)
    bt = i32([list(range(5)), list(range(5, 10))])
    T = 259
    z = i64([0] * T)
    path, acc, new, nxt, err = i32([7] * T), i32([9, 9]), i32([9, 9]), i64([9, 9]), i32([0])
    ffd.ffd_tree_commit(z, z, i32([300, 2]), bt, k, v, path, acc, nxt, new, cu_nodes=i32([0, 257, 259]),
                        error_word=err)
    assert ffd.ffd_get_error(err) == 5
    assert acc.tolist() == [0, 2] and new.tolist() == [300, 2] and nxt.tolist() == [-1, 0]
    assert path.tolist() == [-1] * 257 + [0, 1]


def test_graph_and_values_alone():
    gen = torch.Generator().manual_seed(7)
    bt, P = table([10], [20], gen)
    v0 = torch.randn((P, 4, 64, 128), generator=gen).to(BF16).cuda()
    v = v0.clone()
    par = R.make_parents("random", 20, gen)
    draft, target = tokens(par, 0.9, gen)
    d, t, path = i64(draft), i64(target), i32([0] * 20)
    acc, new, nxt = i32([0]), i32([0]), i64([0])
    lens, tab, parents = i32([30]), bt.cuda(), i32(par)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ffd.ffd_tree_commit(d, t, lens, tab, None, v, path, acc, nxt, new, parents=parents)
    for _ in range(2):
        v.copy_(v0)
        g.replay()
        way = R.accepted_path(d.tolist(), t.tolist(), par)
        assert int(acc[0]) == len(way) and path.tolist()[:len(way)] == way
        page = int(bt[0, 0])
        for to, node in enumerate(way):
            assert torch.equal(v[page, :, 10 + to], v0[page, :, 10 + node])
        t.fill_(99)  # nothing is confirmed the second time
