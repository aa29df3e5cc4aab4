"""Tensors of the speculative step's entries that share memory (no GPU needed): whatever is written over what
another block still reads or writes is refused."""
import ctypes

import pytest
import torch

import sparse_quantized_attention_gb300 as ffd
from sparse_quantized_attention_gb300 import _build
from sparse_quantized_attention_gb300.ffd import RESID_RECORD_BYTES, THUMB_RECORD_BYTES

INVALID, CUDA = 1, 4
FAR = 1 << 24  # between tensors, larger than any here


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ffd.lib()


def places(names):
    return {n: 0x10000000 + i * FAR for i, n in enumerate(names)}


def sharing(at, size, one, other, step):
    """`one` moved so that its first, and so that its last bytes are other's."""
    low = at[other] + max(0, (size[other] - 1) // step * step)
    yield {**at, one: low}
    yield {**at, one: at[other] - max(0, (size[one] - 1) // step * step)}


def pairs(written, read, inplace=()):
    for i, w in enumerate(written):
        for x in read + written[:i]:
            if (w, x) not in inplace:
                yield w, x


# ---- append -------------------------------------------------------------------------------------
T, HQ, HKV, P, B, MB, ROT = 6, 8, 2, 5, 2, 3, 128
ROWS = {"q": HQ, "q_out": HQ, "k_new": HKV, "v_new": HKV}
A_ARGS = ("q", "k_new", "v_new", "freq", "places", "cu", "pos", "bt", "q_out", "k", "v", "thumb", "resid", "err")
A_SIZE = dict(q=T * HQ * 256, q_out=T * HQ * 256, k_new=T * HKV * 256, v_new=T * HKV * 256, freq=2 * ROT, places=4 * T,
              cu=4 * (B + 1), pos=4 * B, bt=4 * B * MB, k=P * HKV * 16384, v=P * HKV * 16384,
              thumb=P * HKV * THUMB_RECORD_BYTES, resid=P * HKV * RESID_RECORD_BYTES, err=4)


def append(lib, at, strides=None, tokens=T):
    s = {n: h * 128 for n, h in ROWS.items()}
    s.update(strides or {})
    p = ffd.RopeParams(B, HQ, HKV, 128, 64, P, MB, 0, tokens, ROT, 0, 1.0, s["q"], s["q_out"], s["k_new"], s["v_new"])
    return lib.ffd_rope_append(ctypes.byref(p), *[at[n] for n in A_ARGS], None)


def goes_on(call):
    """A call that the checks let through: without a GPU it ends at the launch."""
    if not torch.cuda.is_available():  # (the addresses are no memory)
        assert call() == CUDA


@pytest.mark.parametrize("w,x", list(pairs(["q_out", "k", "v", "thumb", "resid", "err"], [
    "q", "k_new", "v_new", "freq", "places", "cu", "pos", "bt"])))
def test_append_refuses(lib, w, x):
    at = places(A_ARGS)
    goes_on(lambda: append(lib, at))
    for moved in sharing(at, A_SIZE, w, x, 4 if w == "err" else 16):
        assert append(lib, moved) == INVALID
    for moved in sharing(at, A_SIZE, x, w, 16 if x in ROWS or x in ("k", "v", "thumb", "resid") else 4):
        assert append(lib, moved) == INVALID


def test_append_between_rows(lib):
    """Rows of one wide buffer: q in place, q_out beside them, and every offset of a tensor against another's."""
    wide = 2 * (HQ + HQ + 2 * HKV) * 128  # bytes: q, a place for q_out, k, v
    at = places(A_ARGS)
    s = {n: wide // 2 for n in ROWS}
    at.update(q=at["q"], q_out=at["q"], k_new=at["q"] + 2 * HQ * 256, v_new=at["q"] + (2 * HQ + HKV) * 256)
    goes_on(lambda: append(lib, at, s))
    beside = {**at, "q_out": at["q"] + HQ * 256}
    goes_on(lambda: append(lib, beside, s))
    for off in range(16, wide, 16):  # q_out of each place in the row, and rows further on or back
        fits = HQ * 256 <= off <= HQ * 256
        for row in (0, 1, -1, T - 1, 1 - T):
            moved = {**at, "q_out": at["q"] + off + row * wide}
            # what rows of q_out there share with rows of q, k_new or v_new
            shared = any(at["q"] + off + (row + i) * wide < at[n] + j * wide + h * 256
                         and at[n] + j * wide < at["q"] + off + (row + i) * wide + HQ * 256
                         for n, h in (("q", HQ), ("k_new", HKV), ("v_new", HKV))
                         for i in range(T) for j in range(T))
            assert not (fits and shared)
            if shared:
                assert append(lib, moved, s) == INVALID, (off, row)
            elif off % 4096 == 0 or row:
                goes_on(lambda: append(lib, moved, s))
    # q in place is q alone: not k_new's or v_new's rows as well
    for n in ("k_new", "v_new"):
        assert append(lib, {**at, n: at["q"]}, s) == INVALID
    # one distance for q_out, another for the rest: not told apart
    assert append(lib, beside, {**s, "q_out": wide}) == INVALID
    # one row has no distance
    one = {**beside, "k_new": at["q"] + HQ * 512, "v_new": at["q"] + HQ * 512 + HKV * 256, "cu": at["cu"]}
    goes_on(lambda: append(lib, one, {**s, "q_out": 8 * HQ * 128}, tokens=1))


# ---- attention ----------------------------------------------------------------------------------
T_ARGS = ("q", "k", "v", "sl", "cu", "par", "bt", "keep", "out", "lse", "ws")


def test_attention_refuses(lib):
    p = ffd.make_tree_params(B, HQ, HKV, P, MB, max_q_len=3, total_q=T, num_splits=2)
    size = dict(q=T * HQ * 256, k=P * HKV * 16384, v=P * HKV * 16384, sl=4 * B, cu=4 * (B + 1), par=4 * T,
                bt=4 * B * MB, keep=B * HKV * MB, out=T * HQ * 256, lse=4 * T * HQ, ws=ffd.ffd_tree_workspace_size(p))
    assert max(size.values()) < FAR
    at = places(T_ARGS)

    def call(at):
        return lib.ffd_tree_attention(ctypes.byref(p), *[at[n] for n in T_ARGS], size["ws"], None)

    goes_on(lambda: call(at))
    align = dict(ws=256, q=16, k=16, v=16, out=16, keep=1)
    for w, x in pairs(["out", "lse", "ws"], ["q", "k", "v", "sl", "cu", "par", "bt", "keep"]):
        for one, other in ((w, x), (x, w)):
            for moved in sharing(at, size, one, other, align.get(one, 4)):
                assert call(moved) == INVALID, (one, other)


# ---- commit -------------------------------------------------------------------------------------
C_ARGS = ("draft", "target", "par", "cu", "sl", "bt", "k", "v", "thumb", "resid", "path", "acc", "nxt", "lens", "err")


def test_commit_refuses(lib):
    size = dict(draft=8 * T, target=8 * T, par=4 * T, cu=4 * (B + 1), sl=4 * B, bt=4 * B * MB,
                k=P * HKV * 16384, v=P * HKV * 16384, thumb=P * HKV * THUMB_RECORD_BYTES,
                resid=P * HKV * RESID_RECORD_BYTES, path=4 * T, acc=4 * B, nxt=8 * B, lens=4 * B, err=4)
    at = places(C_ARGS)
    desc = ffd.CacheDesc(P, HKV, 128, 64)

    def call(at):
        return lib.ffd_tree_commit(ctypes.byref(desc), B, MB, T, *[at[n] for n in C_ARGS], None)

    goes_on(lambda: call(at))
    align = dict(draft=8, target=8, nxt=8, k=16, v=16, thumb=16, resid=16)
    for w, x in pairs(["path", "acc", "nxt", "lens", "k", "v", "thumb", "resid", "err"],
                      ["draft", "target", "par", "cu", "sl", "bt"]):
        for one, other in ((w, x), (x, w)):
            for moved in sharing(at, size, one, other, align.get(one, 4)):
                assert call(moved) == INVALID, (one, other)
