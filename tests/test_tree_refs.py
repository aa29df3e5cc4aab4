"""The 64-bit statements of tests/tree_refs.py against brute force on small cases (CPU)."""
import cmath
import math

import torch

from tests import tree_refs as R


def test_rotation_is_a_complex_turn():
    gen = torch.Generator().manual_seed(0)
    x = torch.randn((3, 2, 128), generator=gen).half()
    f = torch.rand(32, generator=gen)
    places = torch.tensor([0, 7, 100000])
    for inter in (False, True):
        y, _ = R.rotated64(x, places, f, inter, 1.5)
        for t in range(3):
            for i in (0, 5, 31):
                a, b = (2 * i, 2 * i + 1) if inter else (i, i + 32)
                z = complex(float(x[t, 1, a]), float(x[t, 1, b]))
                w = 1.5 * z * cmath.exp(1j * int(places[t]) * float(f[i]))
                assert abs(complex(float(y[t, 1, a]), float(y[t, 1, b])) - w) < 1e-9
        assert torch.equal(y[..., 64:], x[..., 64:].double())


def test_attention_by_hand():
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn((2, 1, 64, 128), generator=gen).half() for _ in range(2))
    q = torch.randn((4, 1, 128), generator=gen).half()
    parents = [-1, 0, 0, 2]
    bt = torch.tensor([[1, 0]], dtype=torch.int32)
    n = 67
    for window in (0, 2, 66):
        out, lse, *_ = R.attention64(q, k, v, [n], [0, 4], bt, parents, window=window)
        sees = {0: [63], 1: [63, 64], 2: [63, 65], 3: [63, 65, 66]}
        depth = [0, 1, 1, 2]
        for i in range(4):
            js = [j for j in range(63) if not window or j > 63 + depth[i] - window]
            js += [j for j in sees[i] if not window or depth[j - 63] > depth[i] - window]
            rows = [(1 if j < 64 else 0, j % 64) for j in js]
            s = [float(q[i, 0].double() @ k[p, 0, r].double()) / math.sqrt(128) for p, r in rows]
            z = math.log(sum(math.exp(x) for x in s))
            assert abs(z - float(lse[i, 0])) < 1e-9
            o = sum(math.exp(x - z) * v[p, 0, r].double() for x, (p, r) in zip(s, rows))
            assert (o - out[i, 0]).abs().max() < 1e-9


def test_path():
    #       0 -> 1 -> 3, 0 -> 2 -> 4, 2 -> 5
    parents = [-1, 0, 0, 1, 2, 2]
    draft = [9, 1, 2, 3, 4, 5]
    assert R.accepted_path(draft, [1, 3, 7, 0, 0, 0], parents) == [0, 1, 3]
    assert R.accepted_path(draft, [2, 3, 5, 0, 0, 0], parents) == [0, 2, 5]
    assert R.accepted_path(draft, [8, 3, 5, 0, 0, 0], parents) == [0]
    # a second root is no path
    assert R.accepted_path([9, 1], [1, 1], [-1, -1]) == [0]
    # of equal depth the lower index
    assert R.accepted_path([9, 5, 5], [5, 0, 0], [-1, 0, 0]) == [0, 1]


def test_trees():
    gen = torch.Generator().manual_seed(2)
    for kind in ("chain", "star", "forest", "binary", "random"):
        p = R.make_parents(kind, 20, gen)
        assert all(-1 <= x < i for i, x in enumerate(p))
        mine, depth = R.related(p)
        assert torch.equal(mine.sum(1) - 1, depth)
