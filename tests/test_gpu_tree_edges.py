"""Tree attention on the GPU where it could go wrong unseen: what a probability is rounded to."""
import pytest
import torch

import sparse_quantized_attention_gb300 as ffd

from tests import tree_refs as R
from tests.test_gpu_rope import i32
from tests.test_gpu_tree import BF16, F16, Problem

pytestmark = pytest.mark.gpu


# ---- probabilities in two parts -----------------------------------------------------------------
def close(out, lse, amax, wabs, usum, dtype):
    """Bound of |library - 64 bits| where a probability enters its product as two numbers of dtype: the first is off
    by half a step, the second, what is left, by half a step of that: 2^-16 of the probability in bf16 and 2^-22 in
    fp16, there 2^-25 where it is below 2^-14, of 2^7 and more for the largest. Scores, powers and sums as in
    tree_refs.tolerance; the products' sums over a page are truncated in eights more additions of 2^-23."""
    ds = amax * 2.0 ** -16
    half = R.half_step(dtype)
    rel = (half ** 2 + 2.0 ** -17 + 2.2 * ds)[..., None]
    least = 2.0 ** -32 if dtype == F16 else 2.0 ** -100
    return half * out.abs() + (rel * wabs + least * usum) * (1 + half) + R.tiny(dtype)


SHAPES = [  # name, Hq, Hkv, lengths, nodes, kind
    ("few", 8, 2, [13, 40], [12, 9], "random"), ("token", 28, 4, [100, 3000], [1, 1], "random"),
    ("one_tile", 8, 2, [700, 300], [16, 32], "random"), ("two_tiles", 8, 2, [40, 700], [40, 61], "random"),
    ("both", 7, 1, [200, 2000], [36, 5], "forest"), ("cut", 8, 1, [20000], [12], "random")]
# more than 2 floor(128 / G) nodes: one part there
GROUPS = [("groups", 7, 1, [200, 2000], [37, 5], "forest"), ("chunk", 8, 1, [300, 2000], [300, 150], None),
          ("most", 8, 1, [256], [256], "binary")]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=[s[0] for s in SHAPES])
@pytest.mark.parametrize("gain", [0.3, 1.0, 4.0])
def test_probabilities_keep_two_parts(shape, dtype, gain):
    """out is the 64-bit result but for its own rounding and what scores and sums are off by."""
    _, Hq, Hkv, lens, nqs, kind = shape
    x = Problem(Hq, Hkv, lens, nqs, dtype, kind, seed=41, gain=gain)
    got, _ = x.run()
    ref = R.attention64(x.q, x.k, x.v, lens, x.cu, x.bt, x.parents)
    mine = ~torch.isnan(ref[1])
    over = ((got.double() - ref[0]).abs() - close(*ref, dtype))[mine]
    assert float(over.max()) <= 0, (float(over.max()), int((over > 0).sum()), over.numel())


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES + GROUPS, ids=[s[0] for s in SHAPES + GROUPS])
@pytest.mark.parametrize("gain", [1.0, 4.0, 16.0])
def test_one_value_comes_back(shape, dtype, gain):
    """Every V the same number: whatever the probabilities are, the result is that number. Numerator and denominator
    differ by the parts' 2^-16 (where there is one part, by nothing: O is divided by the sum of what was multiplied) and
    by the sums' roundings, 2^-14 together over these lengths; the number just below 2 has half a step of 2^-9 of
    itself (bf16) or 2^-12 to either side."""
    _, Hq, Hkv, lens, nqs, kind = shape
    x = Problem(Hq, Hkv, lens, nqs, dtype, kind, seed=42, gain=gain)
    one = 2.0 - torch.finfo(dtype).eps
    x.v.fill_(one)
    got, _ = x.run()
    assert bool((got[:x.T] == one).all()), int((got[:x.T] != one).sum())


# ---- waits that run out -------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("splits", [0, 3, 40])
@pytest.mark.parametrize("nq", [1, 20, 60, 100])
def test_a_wait_for_other_parts_runs_out(nq, splits, dtype):
    """The counts of published parts begin at large negative numbers, so that CTAs that share an item wait for
    what never comes: each gives up at its limit, 1 ms, is drained at once (what it had under way has landed) and
    the call reports it. On a workspace filled with zeros again the next call gives what it gave before."""
    x = Problem(8, 2, [9000, 100, 2500], [nq] * 3, dtype, seed=nq)
    want = x.run(num_splits=splits)
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    p = x.params(num_splits=splits, wait_limit_us=1000)
    args = (x.q, x.k, x.v, i32(x.lens), x.bt.cuda(), torch.empty_like(want[0]), x.ws)
    more = dict(parents=i32(x.parents), cu_q=i32(x.cu))
    for _ in range(3):
        x.ws.fill_(0x80)
        x.ws[:256].zero_()  # the error word
        e0.record()
        ffd.ffd_tree_attention(p, *args, **more)
        e1.record()
        assert ffd.ffd_get_error(x.ws) == 7
        assert 1.0 <= e0.elapsed_time(e1) < 500.0  # ms: no drain ran to its own bound
        x.ws.zero_()
        again = x.run(num_splits=splits)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
