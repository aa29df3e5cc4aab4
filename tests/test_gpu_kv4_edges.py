"""The 4-bit cache's attention where its arithmetic, its inputs or its plan come to an edge. Bounds as
in tests/kv4_refs.py."""
import math
import os
import subprocess
import sys

import pytest
import torch

import sparse_quantized_attention_gb300 as ffd
from tests import kv4_refs as R
from tests.test_gpu_kv4 import BF16, F16, Case, i32, offsets, table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("octave", [22, 23, 24, 25, 26, 27])
@pytest.mark.parametrize("nq", [1, 3, 40])
def test_scores_past_2_to_the_24(nq, octave, dtype):
    """Scores of 2^octave (log2 units) whose largest grows by a little from page to page: where fp32 holds
    no reference that much below or above them, no probability may leave f16's range. All V rows are
    alike, so a row's output is its V whatever the weights: each product and the sum l carry at most
    f16's half step, 2^-11, or 2^-25 of probabilities of which the largest is at least 1."""
    G, B, n = 8, 4, 64 * 64
    gen = torch.Generator().manual_seed(octave)
    bt, P = table([n] * B, gen)
    # every token's K is (16384, 0, ..); the first of each page has one of 5 codes in channel 1
    k = torch.zeros((B, n, 1, 128))
    k[..., 0] = 16384.0
    k[:, ::64, 0, 1] = 1092.0 * (torch.arange(n // 64) % 5)
    v = torch.randn((1, 1, 1, 128), generator=gen).expand(B, n, 1, 128)
    cache = ffd.alloc_kv4_cache(P, 1)
    ffd.ffd_kv4_write(k.to(F16).reshape(-1, 1, 128).cuda(), v.to(F16).reshape(-1, 1, 128).cuda(),
                      i32([0] * B), bt.cuda(), cache)
    unit = math.log2(math.e) / math.sqrt(128)  # log2 units of a score
    q = torch.zeros((B * nq, G, 128))
    rows = B * nq * G
    q[..., 0] = 2.0 ** octave * torch.linspace(1.0, 1.9, rows).reshape(-1, G) / (16384 * unit)
    q[..., 1] = torch.linspace(0.5, 24.0, rows).reshape(-1, G).flip(0) / (1092 * unit)
    q = q.clamp(max=65504.0).to(dtype).cuda()
    for splits in (B, 0):
        p = ffd.make_kv4_params(B, G, 1, P, bt.shape[1], max_q_len=nq, dtype=dtype, num_splits=splits)
        ws = ffd.alloc_kv4_workspace(p)
        out = torch.empty_like(q)
        lse = torch.empty((B * nq, G), device="cuda")
        ffd.ffd_kv4_attention(p, q, cache, i32([n] * B), bt.cuda(), out, ws, lse=lse)
        assert ffd.ffd_get_error(ws) == 0
        assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
        want = R.held64(v[0, 0, 0].to(F16)).cuda()
        half = torch.finfo(dtype).eps / 2
        rel = half + (1 + half) * (2.0 ** -11 + n * 2.0 ** -25 + 2.0 ** -18)
        assert bool(((out.double() - want).abs() <= rel * want.abs() + 2.0 ** -25).all())
    ref = R.attention64(q, cache.k4, cache.v4, [n] * B, offsets([nq] * B), bt, 1, sm=float(p.sm_scale))
    tol = R.tolerance(*ref, dtype)[1]
    assert bool(((lse.double() - ref[1]).abs() <= tol).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 60000.0])
@pytest.mark.parametrize("nq,window", [(4, 0), (100, 0), (1, 40), (6, 40), (100, 40)])
def test_a_token_out_of_range_reaches_only_rows_that_see_it(nq, window, bad):
    """The rows before it, and those whose window has passed it, are what they are without it."""
    gen = torch.Generator().manual_seed(nq + window)
    Hkv, G, n = 2, 4, 300
    at = n - (45 if nq <= 6 and window else min(nq, 60) // 2 + 1)  # the token, in the last two pages
    bt, P = table([n], gen)
    x = torch.randn((2, n, Hkv, 128), generator=gen).to(F16)
    q = torch.randn((nq, Hkv * G, 128), generator=gen).to(F16).cuda()
    p = ffd.make_kv4_params(1, Hkv * G, Hkv, P, bt.shape[1], max_q_len=nq, dtype=F16, window=window)
    cache = ffd.alloc_kv4_cache(P, Hkv)
    ffd.ffd_kv4_write(x[0].cuda(), x[1].cuda(), i32([0]), bt.cuda(), cache)
    ref = R.attention64(q, cache.k4, cache.v4, [n], [0, nq], bt, Hkv, window=window,
                        sm=float(p.sm_scale))
    tol, tol_lse = R.tolerance(*ref, F16)
    x[0, at, 0, 5] = bad
    x[1, at, :, 77] = bad
    err = i32([0])
    ffd.ffd_kv4_write(x[0].cuda(), x[1].cuda(), i32([0]), bt.cuda(), cache, error_word=err)
    assert ffd.ffd_get_error(err) == 6
    ws = ffd.alloc_kv4_workspace(p)
    out, lse = torch.empty_like(q), torch.empty((nq, Hkv * G), device="cuda")
    ffd.ffd_kv4_attention(p, q, cache, i32([n]), bt.cuda(), out, ws, lse=lse)
    assert ffd.ffd_get_error(ws) == 0
    pos = torch.arange(n - nq, n, device="cuda")
    blind = (pos < at) | ((pos - window >= at) if window else (pos < 0))
    assert bool(blind.any())
    assert bool(((out.double() - ref[0]).abs() <= tol)[blind].all())
    assert bool(((lse.double() - ref[1]).abs() <= tol_lse)[blind].all())
    held = torch.empty((2, n, Hkv, 128), dtype=F16, device="cuda")
    ffd.ffd_kv4_read(cache, i32([0]), bt.cuda(), held[0], held[1])
    assert bool(torch.isfinite(held).all())


@pytest.mark.parametrize("nq", [1, 3, 6, 20, 100])
@pytest.mark.parametrize("window", [1, 40, 64, 130])
def test_tokens_behind_every_window_may_be_anything(nq, window):
    """A page at the window's edge may hold tokens that were never written (a long prompt of which only
    the part that the window reaches was)."""
    lens = [300, 64, 1000, 65]
    c = Case(lens, [min(nq, n) for n in lens], 2, 4, window=window, seed=nq + window)
    c.poison_unused()
    for b, n in enumerate(lens):
        for t in range(0, max(0, n - c.qlens[b] - window + 1)):
            page = int(c.bt[b, t // 64])
            for rec in (c.k4, c.v4):
                rec[page, :, 4096 + 16 * (t % 64):4112 + 16 * (t % 64)] = 0xff
    out, lse = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("q", [1, 3, 6, 40, 400])
@pytest.mark.parametrize("splits", [0, 3])
def test_a_wait_that_runs_out(q, splits):
    """The shortest limit, below the time of a copy: the call ends, reports it or is right, and leaves the
    workspace to the next call. (The time of a call is bounded: nothing waits for what never comes.)"""
    c = Case([9000, 100, 2500], [q, min(q, 100), q], 2, 4, seed=q)
    p, short = c.params(num_splits=splits), c.params(num_splits=splits, wait_limit_us=1)
    ws = ffd.alloc_kv4_workspace(p)
    good = c.buffers()
    c.call(*good, ws, p)
    assert ffd.ffd_get_error(ws) == 0
    c.check(*good)
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(20):
        out, lse = c.buffers()
        e0.record()
        c.call(out, lse, ws, short)
        e1.record()
        status = ffd.ffd_get_error(ws)
        assert e0.elapsed_time(e1) < 1500.0  # ms; a drain may take 2 s when its copy never lands
        assert status in (0, 7)
        if status == 0:
            assert torch.equal(out, good[0])
        out, lse = c.buffers()
        c.call(out, lse, ws, p)
        assert ffd.ffd_get_error(ws) == 0
        assert torch.equal(out, good[0]) and torch.equal(lse, good[1])


@pytest.mark.parametrize("lens,q", [([32768] + [1024] * 18, 9), ([700] * 37 + [16384], 64),
                                    ([300, 9000] + [200] * 80, 30)])
def test_unequal_lengths_are_cut(lens, q):
    """One long sequence among short ones, as many units as there are SMs or more: its items are not
    left to a few CTAs. The same call with cut items forced takes about as long (it took a sixth)."""
    c = Case(lens, [q] * len(lens), 8, 4, seed=len(lens))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    times = []
    for splits in (0, sms):
        p = c.params(num_splits=splits)
        ws = ffd.alloc_kv4_workspace(p)
        out, lse = c.buffers()
        best = math.inf
        for _ in range(8):
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda._sleep(1_000_000)  # the host is ahead when the first event is reached
            e0.record()
            c.call(out, lse, ws, p)
            e1.record()
            torch.cuda.synchronize()
            best = min(best, e0.elapsed_time(e1))
        assert ffd.ffd_get_error(ws) == 0
        c.check(out, lse)
        times.append(best)
    assert times[0] < 2.0 * times[1]


@pytest.mark.parametrize("q", [1, 2, 6, 20, 90])
def test_bad_offsets_and_lengths_of_any_row_count(q):
    """A sequence whose offsets are out of order keeps its rows as they were, one whose length is out of
    range is clamped; the others are what they are."""
    lens = [300, 200, 100]
    c = Case(lens, [q] * 3, 2, 4, seed=q, tail=3)
    cache, T = ffd.Kv4Cache(c.k4, c.v4), c.T
    p = c.params()
    ws = ffd.alloc_kv4_workspace(p)

    def check(lens, cu, good):
        out, lse = c.buffers()
        ffd.ffd_kv4_attention(p, c.q, cache, i32(lens), c.bt, out, ws, cu_q=i32(cu), lse=lse)
        assert ffd.ffd_get_error(ws) == 5
        mine = torch.zeros(T, dtype=torch.bool, device="cuda")
        for b in good:
            n, t0, t1 = min(max(lens[b], 0), 64 * c.bt.shape[1]), cu[b], cu[b + 1]
            mine[t0:t1] = True
            ref = R.attention64(c.q[t0:t1], c.k4, c.v4, [n], [0, t1 - t0], c.bt[b:b + 1], 2,
                                sm=float(p.sm_scale))
            tol, tol_lse = R.tolerance(*ref, BF16)
            sees = ref[1] > -math.inf
            assert bool(((out[t0:t1].double() - ref[0]).abs() <= tol)[sees].all())
            assert bool(((lse[t0:t1].double() - ref[1]).abs() <= tol_lse)[sees].all())
            assert bool((out[t0:t1][~sees] == 0).all())
            assert bool((lse[t0:t1][~sees] == -math.inf).all())
        assert bool((out[~mine] == 3.0).all()) and bool((lse[~mine] == 3.0).all())

    check(lens, [0, q, T + 1, 2 * q], [0])          # an end past total_q, then offsets that fall
    check(lens, [-1, q, 2 * q, 3 * q], [1, 2])
    check(lens, [0, q, 2 * q + 1, 3 * q], [0, 2])   # one row more than max_q_len
    check([300, -5, 100], c.cu, [0, 1, 2])
    check([300, 2 ** 31 - 1, 100], c.cu, [0, 1, 2])  # clamped; its pages past the table are dropped


@pytest.mark.parametrize("q,G", [(3, 4), (6, 4), (4, 8), (20, 4), (90, 8)])
def test_a_bad_query_stays_in_its_row(q, G):
    c = Case([500, 300], [q, q], 2, G, seed=q)
    good, good_lse = c.run()
    bad = [(0, 3, math.nan), (q - 1, 2 * G - 1, math.inf), (q, 0, -math.inf), (2 * q - 1, G, math.nan)]
    for t, h, x in bad:
        c.q[t, h, 17] = x
    out, lse = c.run()
    same = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    for t, h, x in bad:
        assert not bool(torch.isfinite(out[t, h]).all())
        same[t, h] = False
    assert torch.equal(out[same], good[same]) and torch.equal(lse[same], good_lse[same])


FIRST_CALL = """
import torch
import sparse_quantized_attention_gb300 as ffd
B, Hkv, G, n, P = 2, 2, 4, 130, 8
gen = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn((2, B * n, Hkv, 128), generator=gen, device="cuda").bfloat16()
bt = torch.arange(6, dtype=torch.int32, device="cuda").reshape(B, 3)
first = torch.zeros(B, dtype=torch.int32, device="cuda")
lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
cache = ffd.alloc_kv4_cache(P, Hkv)
back = torch.empty_like(x)
calls = []
for nq in (1, 3, 5, 8, 40):
    p = ffd.make_kv4_params(B, Hkv * G, Hkv, P, 3, max_q_len=nq)
    q = torch.randn((B * nq, Hkv * G, 128), generator=gen, device="cuda").bfloat16()
    calls.append((p, q, torch.empty_like(q), ffd.alloc_kv4_workspace(p)))

def run():
    ffd.ffd_kv4_write(x[0], x[1], first, bt, cache)
    ffd.ffd_kv4_read(cache, first, bt, back[0], back[1])
    for p, q, out, ws in calls:
        ffd.ffd_kv4_attention(p, q, cache, lens, bt, out, ws)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
graph.replay()
torch.cuda.synchronize()
got = [back.clone()] + [c[2].clone() for c in calls]
for t in [back] + [c[2] for c in calls]:
    t.zero_()
run()
assert all(torch.equal(a, b) for a, b in zip(got, [back] + [c[2] for c in calls]))
assert all(ffd.ffd_get_error(c[3]) == 0 for c in calls)
"""


def test_a_first_call_may_be_captured():
    """Every kernel is called for the first time in its process under a graph's capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("q", [1, 3, 20, 100])
@pytest.mark.parametrize("kw", [dict(window=150, keep=0.5), dict(window=2 ** 31 - 1),
                                dict(window=2 ** 31 - 1, keep=0.3)],
                         ids=["window_mask", "largest_window", "largest_window_mask"])
def test_windows(q, kw):
    """A window and a mask together; a window as large as can be named, with more queries than tokens."""
    c = Case([1000, 65, 2, 0], [q] * 4, 2, 4, seed=q, **kw)
    c.poison_unused()
    out, lse = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("B", [1, 3, 100, 700])
@pytest.mark.parametrize("q", [1, 3, 20])
def test_nothing_to_see(q, B):
    """Empty sequences alone, and one token among them."""
    for last in (0, 1):
        c = Case([0] * (B - 1) + [last], [q] * B, 2, 4, seed=q)
        out, lse = c.run()
        c.check(out, lse)


def test_offsets_out_of_order_write_inside_the_cache():
    """cu_tokens that fall and pass the rows' number: rows go where they name a place or nowhere."""
    gen = torch.Generator().manual_seed(1)
    Hkv, T, width = 2, 12, 2
    bt, P = table([128, 128, 128], gen, spare=2)
    x = torch.randn((T, Hkv, 128), generator=gen).to(BF16).cuda()
    cache = ffd.alloc_kv4_cache(P, Hkv)
    used = set(bt.flatten().tolist())
    spare = [i for i in range(P) if i not in used]
    for t in cache:
        t.fill_(9)
    err = i32([0])
    for cu in ([0, 9, 3, 12], [5, 2, 1, 0], [-8, 4, 100, 20], [20, 30, 40, 50]):
        ffd.ffd_kv4_write(x, x, i32([0, 60, 126]), bt.cuda(), cache, cu_tokens=i32(cu), error_word=err)
        assert ffd.ffd_get_error(err) in (0, 5)
        out = torch.full_like(x, 5.0)
        ffd.ffd_kv4_read(cache, i32([0, 60, 126]), bt.cuda(), out, None, cu_tokens=i32(cu),
                         error_word=err)
        assert ffd.ffd_get_error(err) in (0, 5)
    assert all(bool((t[spare] == 9).all()) for t in cache)
