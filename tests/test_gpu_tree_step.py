"""A speculative step's calls one after another, as a program makes them: append, attend, commit, and a
plain decode step over the cache that they leave."""
import math

import pytest
import torch

import sparse_quantized_attention_gb300 as ffd
from tests import tree_refs as R
from tests.test_gpu_rope import frequencies, i32, near

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("graphed", [False, True])
def test_steps_together(graphed):
    gen = torch.Generator().manual_seed(3)
    B, Hq, Hkv, nq, width = 3, 8, 2, 13, 8
    P = B * width
    bt = torch.randperm(P, generator=gen).to(torch.int32).reshape(B, width).cuda()
    k = torch.zeros((P, Hkv, 64, 128), dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    cache = ffd.alloc_quantized_cache(P, Hkv)
    freq = frequencies(128).cuda()
    lens = [150, 63, 1]
    err = i32([0])
    # prompts
    x = torch.randn((sum(lens), Hq + 2 * Hkv, 128), generator=gen).to(BF16).cuda()
    cu = [0, 150, 213, 214]
    qkv = (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])
    out = torch.empty((sum(lens), Hq, 128), dtype=BF16, device="cuda")
    ffd.ffd_rope_append(*qkv, freq, i32([0] * B), bt, out, k, v, cu_tokens=i32(cu), quantized=cache,
                        error_word=err)
    history = [(qkv[1][cu[b]:cu[b + 1]], qkv[2][cu[b]:cu[b + 1]]) for b in range(B)]

    # buffers of a step
    T = B * nq
    y = torch.zeros((T, Hq + 2 * Hkv, 128), dtype=BF16, device="cuda")
    q, kn, vn = y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]
    qr = torch.empty((T, Hq, 128), dtype=BF16, device="cuda")
    att, lse = torch.empty_like(qr), torch.empty((T, Hq), device="cuda")
    first, n, new = i32(lens), i32([0] * B), i32([0] * B)
    places, par = i32([0] * T), i32([0] * T)
    draft = torch.zeros(T, dtype=torch.int64, device="cuda")
    target = torch.zeros_like(draft)
    path, acc = i32([0] * T), i32([0] * B)
    nxt = torch.zeros(B, dtype=torch.int64, device="cuda")
    p = ffd.make_tree_params(B, Hq, Hkv, P, width, max_q_len=nq)
    ws = ffd.alloc_tree_workspace(p)

    def step():
        ffd.ffd_rope_append(q, kn, vn, freq, first, bt, qr, k, v, rope_positions=places, quantized=cache,
                            error_word=err)
        ffd.ffd_tree_attention(p, qr, k, v, n, bt, att, ws, parents=par, lse=lse)
        ffd.ffd_tree_commit(draft, target, n, bt, k, v, path, acc, nxt, new, parents=par, quantized=cache,
                            error_word=err)
        first.copy_(new)

    graph = None
    for turn in range(6):
        parents, depths, toks, tgts = [], [], [], []
        for b in range(B):
            up = R.make_parents("random", nq, gen)
            d = torch.randint(0, 9, (nq,), generator=gen).tolist()
            t = [9] * nq
            for i in range(1, nq):
                if float(torch.rand(1, generator=gen)) < 0.7:
                    t[up[i]] = d[i]
            parents, toks, tgts = parents + up, toks + d, tgts + t
            depths += R.related(up)[1].tolist()
        y.copy_(torch.randn(y.shape, generator=gen).to(BF16))
        before = first.tolist()
        n.copy_(first + nq)
        places.copy_(i32([before[i // nq] + depths[i] for i in range(T)]))
        par.copy_(i32(parents))
        draft.copy_(torch.tensor(toks))
        target.copy_(torch.tensor(tgts))
        if graphed and turn > 0:
            if graph is None:
                keep = [t.clone() for t in (k, v, *cache, first)]
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
                for t, old in zip((k, v, *cache, first), keep):
                    assert torch.equal(t, old)      # capturing runs nothing
            graph.replay()
        else:
            step()
        assert ffd.ffd_get_error(err) == 0 and ffd.ffd_get_error(ws) == 0
        # each accepted path from scratch: rotated keys, attention over them, and what is kept
        for b in range(B):
            at = b * nq
            way = R.accepted_path(toks[at:at + nq], tgts[at:at + nq], parents[at:at + nq])
            assert path[at:at + nq].tolist() == way + [-1] * (nq - len(way))
            assert int(nxt[b]) == tgts[at + way[-1]] and int(first[b]) == before[b] + len(way)
            rows = [at + w for w in way]
            history[b] = tuple(torch.cat((h, z[rows])) for h, z in zip(history[b], (kn, vn)))
            size = before[b] + len(way)
            where = torch.arange(size).cuda()
            held = k[bt[b, where // 64].long(), :, where % 64]
            want, bound = R.rotated64(history[b][0], where, freq.cpu())
            near(held, want, bound, "k")
            assert torch.equal(v[bt[b, where // 64].long(), :, where % 64], history[b][1])
            # the path's rows attend as a chain would
            pages, each = bt[b:b + 1].cpu(), len(way)
            ref = R.attention64(qr[rows], k, v, [size], [0, each], pages, None)
            tol, ltol = R.tolerance(*ref, BF16)
            assert bool(((att[rows].double() - ref[0]).abs() <= tol).all())
            assert bool(((lse[rows].double() - ref[1]).abs() <= ltol).all())
    # the records have moved along: a decode step over them is one over the keys that are there
    want = ffd.alloc_quantized_cache(P, Hkv)
    ffd.ffd_quantize_keys(k, want)
    for b in range(B):
        where = torch.arange(int(first[b])).cuda()
        pg, r = bt[b, where // 64].long(), where % 64
        for mine, fresh in zip(cache, want):
            codes = mine.shape[-1] // (68 if mine.shape[-1] > 5000 else 48) * (64 if mine.shape[-1] > 5000 else 32)
            per = codes // 64
            a, c = (z[..., :codes].unflatten(-1, (64, per)) for z in (mine, fresh))
            assert torch.equal(a[pg, :, r], c[pg, :, r])
            a, c = (z[..., codes:].unflatten(-1, (-1, 64, 8)) for z in (mine, fresh))
            assert torch.equal(a[pg, :, :, r], c[pg, :, :, r])
    dp = ffd.make_params(B, Hq, Hkv, P, width, sink=64, local=64, delta=math.inf)
    o = torch.empty((B, Hq, 128), device="cuda")
    one = torch.randn((B, Hq, 128), generator=gen).to(BF16).cuda()
    ffd.ffd_decode_attention(dp, one, cache, v, first, bt, o, ffd.alloc_workspace(dp))
    dense = torch.empty_like(o)
    ffd.ffd_dense_decode(dp, one, k, v, first, bt, dense, ffd.alloc_workspace(dp, dense=True))
    tree = ffd.make_tree_params(B, Hq, Hkv, P, width)
    single = torch.empty((B, Hq, 128), dtype=BF16, device="cuda")
    ffd.ffd_tree_attention(tree, one, k, v, first, bt, single, ffd.alloc_tree_workspace(tree))
    ref = R.attention64(one, k, v, first.tolist(), list(range(B + 1)), bt.cpu(), None)
    tol, _ = R.tolerance(*ref, BF16)
    assert bool(((single.double() - ref[0]).abs() <= tol).all())
    assert float((dense.double() - ref[0]).abs().max()) < 2e-3
    assert float((o.double() - ref[0]).abs().max()) < 0.05   # 8-bit keys
