"""The shortest wait limit (1 us, below the time of a copy) in the kernels whose CTAs wait for nothing but
their own copies: a call ends at once and reports it or is right, waits for its copies before it leaves, and
the next call with the default limit gives what it gave before."""
import pytest
import torch

import ffd_synth
import sparse_quantized_attention_gb300 as ffd
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu


def _params(inp, limit):
    p = H.params_for(inp, 5.0)
    p.wait_limit_us = limit
    return p


def _alternate(call, ws, state):
    """call(limit) writes the tensors `state`; 20 short calls, each followed by an ordinary one."""
    call(0)
    assert ffd.ffd_get_error(ws) == 0
    good = [t.clone() for t in state]
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(20):
        e0.record()
        call(1)
        e1.record()
        status = ffd.ffd_get_error(ws)
        assert e0.elapsed_time(e1) < 1500.0  # ms: no drain waited for what never comes (2 s)
        assert status in (0, 7)
        if status == 0:
            assert all(torch.equal(t, g) for t, g in zip(state, good))
        call(0)
        assert ffd.ffd_get_error(ws) == 0
        assert all(torch.equal(t, g) for t, g in zip(state, good))


@pytest.fixture(scope="module")
def setup():
    w = ffd_synth.custom(2, 8, 2, 3000, sink=64, local=256, seed=21)
    inp = ffd_synth.make_inputs(w)
    dev = H.to_device(inp)
    return inp, dev, H.quantize(dev)


def test_art(setup):
    inp, dev, qc = setup
    w = inp.workload
    ws = ffd.alloc_art_workspace(_params(inp, 0))
    out = torch.empty((w.batch, w.num_q_heads, 128), device="cuda")
    used = torch.empty((w.batch, w.num_kv_heads), dtype=torch.int32, device="cuda")

    def call(limit):
        ffd.ffd_art_attention(_params(inp, limit), 0.0, 0.0, 2, dev["q"], qc, dev["v"],
                              dev["seq_lens"], dev["block_table"], out, ws, blocks_used=used)
    _alternate(call, ws, (out, used))


@pytest.mark.parametrize("selector,budget", [(ffd.SELECT_TOPK, 12), (ffd.SELECT_TOPP, 0.8)])
def test_selectors(setup, selector, budget):
    inp, dev, qc = setup
    w = inp.workload
    ws = ffd.alloc_select_workspace(_params(inp, 0))
    mask = torch.empty((w.batch, w.num_kv_heads, inp.max_blocks), dtype=torch.uint8, device="cuda")

    def call(limit):
        ffd.ffd_select_blocks(_params(inp, limit), selector, budget, dev["q"], qc, dev["seq_lens"],
                              dev["block_table"], mask, ws)
    _alternate(call, ws, (mask,))
