"""Refusals of the speculative step's entries (no GPU needed): bad arguments come back as a status, or
as an FFDError from the binding, before anything is enqueued."""
import ctypes
import math

import pytest
import torch

import sparse_quantized_attention_gb300 as ffd
from sparse_quantized_attention_gb300 import _build
from tests.test_kv4_host import OnGpu

FAKE = 0x100000  # never dereferenced: every call here fails validation first


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ffd.lib()


def test_exports(lib):
    raw = ctypes.CDLL(_build.LIB)
    for name in ("ffd_rope_append", "ffd_tree_workspace_size", "ffd_tree_attention", "ffd_tree_commit"):
        assert hasattr(raw, name)


# ---- append -------------------------------------------------------------------------------------
ROPE = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=64, num_pages=5,
            max_blocks_per_seq=3, dtype=0, total_tokens=6, rot_dim=128, interleaved=0, rot_scale=1.0,
            q_stride=1024, q_out_stride=1024, k_stride=256, v_stride=256)


def append(lib, **kw):
    # q, k_new, v_new, inv_freq, rope_positions, cu, positions, table, q_out, k, v, thumb, resid, error
    ptr = dict(q=FAKE, k_new=FAKE, v_new=FAKE, freq=FAKE, places=None, cu=FAKE, pos=FAKE, bt=FAKE,
               q_out=FAKE, k=FAKE, v=FAKE, thumb=None, resid=None, err=None)
    ptr.update({n: kw.pop(n) for n in list(kw) if n in ptr})
    p = ffd.RopeParams(**{**ROPE, **kw})
    return lib.ffd_rope_append(ctypes.byref(p), *ptr.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 1), (dict(num_q_heads=-1), 1), (dict(num_q_heads=0), 1), (dict(num_kv_heads=0), 1),
    (dict(num_pages=0), 1), (dict(max_blocks_per_seq=0), 1), (dict(total_tokens=-1), 1),
    (dict(dtype=2), 1), (dict(rot_dim=-16), 1), (dict(rot_dim=8), 1), (dict(rot_dim=144), 1),
    (dict(interleaved=2), 1), (dict(rot_scale=math.nan), 1), (dict(rot_scale=math.inf), 1),
    (dict(freq=None), 1), (dict(cu=None, total_tokens=5), 1), (dict(q=None), 1), (dict(q_out=None), 1),
    (dict(v=None), 1), (dict(k=None), 1), (dict(k_new=None), 1), (dict(v_new=None), 1),
    (dict(thumb=FAKE), 1), (dict(resid=FAKE), 1), (dict(pos=None), 1), (dict(bt=None), 1),
    (dict(q_stride=1016), 1), (dict(q_out_stride=1028), 1), (dict(k_stride=128), 1),
    (dict(v_stride=260), 1), (dict(q=FAKE + 8), 1), (dict(k=FAKE + 2), 1), (dict(v_new=FAKE + 4), 1),
    (dict(freq=FAKE + 2), 1), (dict(err=FAKE + 1), 1), (dict(places=FAKE + 2), 1),
    (dict(head_dim=64), 2), (dict(page_size=32), 2), (dict(max_blocks_per_seq=1 << 26), 2),
    (dict(thumb=FAKE, resid=FAKE, dtype=1), 2),
    (dict(num_q_heads=70000, q_stride=70000 * 128, q_out_stride=70000 * 128), 2),
    (dict(q_out=FAKE + 1024), 1),                      # over other rows of q
    (dict(q_stride=2048), 1),                          # in place, but at another distance
])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status


def test_append_of_nothing(lib):
    none = dict(q=None, q_out=None, k_new=None, v_new=None)
    assert append(lib, total_tokens=0, num_q_heads=0, **none) == 0
    assert append(lib, total_tokens=0) == 0
    assert lib.ffd_rope_append(None, *[FAKE] * 14, None) == 1


# ---- attention ----------------------------------------------------------------------------------
def params(**kw):
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, num_pages=10, max_blocks_per_seq=5,
                max_q_len=3, total_q=6, num_splits=2)
    base.update(kw)
    return ffd.make_tree_params(*[base.pop(n) for n in (
        "batch", "num_q_heads", "num_kv_heads", "num_pages", "max_blocks_per_seq")], **base)


def attend(lib, p, ws_bytes=1 << 40, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, sl=FAKE, cu=FAKE, par=FAKE, bt=FAKE, keep=None, out=FAKE, lse=None,
             ws=FAKE)
    a.update(kw)
    return lib.ffd_tree_attention(ctypes.byref(p) if p else None, *a.values(), ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 1), (dict(num_q_heads=7), 1), (dict(num_q_heads=18), 2), (dict(num_pages=0), 1),
    (dict(max_blocks_per_seq=0), 1), (dict(max_blocks_per_seq=1 << 26), 2), (dict(max_q_len=0), 1),
    (dict(total_q=0), 1), (dict(window=-1), 1), (dict(num_splits=-1), 1), (dict(wait_limit_us=-1), 1),
    (dict(sm_scale=0.0), 1), (dict(sm_scale=math.nan), 1), (dict(sm_scale=math.inf), 1),
    (dict(q_stride=8), 1), (dict(q_stride=1028), 1), (dict(batch=40000), 2),
    (dict(num_pages=1 << 25), 2), (dict(max_q_len=1 << 27), 2),
    (dict(max_blocks_per_seq=1 << 24, batch=200, total_q=600), 2),
])
def test_attention_refuses_params(lib, kw, status):
    p = params(**kw)
    assert attend(lib, p) == status
    assert ffd.ffd_tree_workspace_size(p) == 0


def test_attention_refuses_walks_past_int32(lib):
    """B Hkv (blocks + 9) stays below INT32_MAX - 4096: shares of items may end behind the last page."""
    shape = dict(batch=64, num_q_heads=1, num_kv_heads=1, max_q_len=1, total_q=64)
    assert ffd.ffd_tree_workspace_size(params(max_blocks_per_seq=33554422, **shape)) == 0
    assert ffd.ffd_tree_workspace_size(params(max_blocks_per_seq=33554300, **shape)) > 0


def test_attention_refuses_shapes_and_pointers(lib):
    p = params()
    need = ffd.ffd_tree_workspace_size(p)
    assert need > 0 and need % 256 == 0
    for field, value, status in (("head_dim", 64, 2), ("page_size", 16, 2), ("dtype", 3, 1)):
        bad = params()
        setattr(bad, field, value)
        assert attend(lib, bad) == status
    assert attend(lib, None) == 1
    for key in ("q", "k", "v", "sl", "bt", "out", "ws"):
        assert attend(lib, p, **{key: None}) == 1, key
    for key, off in (("q", 8), ("k", 4), ("v", 8), ("out", 2), ("ws", 16), ("cu", 2), ("sl", 1),
                     ("lse", 2), ("par", 2), ("bt", 1)):
        assert attend(lib, p, **{key: FAKE + off}) == 1, key
    far = dict(out=FAKE + (1 << 20))
    assert attend(lib, p, ws_bytes=need - 1, **far) == 3
    assert attend(lib, params(total_q=5), cu=None, **far) == 1   # rows not max_q_len each
    assert attend(lib, params(max_q_len=257, total_q=514), **far) == 2  # a tree of more than 256 nodes
    # q and out are 6 rows of 8 heads: 12288 bytes each
    assert attend(lib, p) == 1
    assert attend(lib, p, out=FAKE + 12288 - 16) == 1
    assert attend(lib, p, q=FAKE + 12288 - 16) == 1


# ---- commit -------------------------------------------------------------------------------------
def commit(lib, desc=(4, 2, 128, 64), batch=2, mb=3, total=6, **kw):
    a = dict(draft=FAKE, target=FAKE, par=FAKE, cu=FAKE, sl=FAKE, bt=FAKE, k=FAKE, v=FAKE, thumb=None,
             resid=None, path=FAKE, acc=FAKE, nxt=FAKE, lens=FAKE + 64, err=None)
    a.update(kw)
    d = ctypes.byref(ffd.CacheDesc(*desc)) if desc else None
    return lib.ffd_tree_commit(d, batch, mb, total, *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(desc=None), 1), (dict(desc=(0, 2, 128, 64)), 1), (dict(desc=(4, 0, 128, 64)), 1),
    (dict(desc=(4, 2, 64, 64)), 2), (dict(desc=(4, 2, 128, 16)), 2), (dict(batch=0), 1),
    (dict(mb=0), 1), (dict(mb=1 << 26), 2), (dict(total=-1), 1), (dict(cu=None, total=5), 1),
    (dict(cu=None, total=514), 2), (dict(draft=None), 1), (dict(target=None), 1), (dict(path=None), 1),
    (dict(sl=None), 1), (dict(bt=None), 1), (dict(acc=None), 1), (dict(nxt=None), 1), (dict(lens=None), 1),
    (dict(thumb=FAKE), 1), (dict(resid=FAKE), 1), (dict(draft=FAKE + 4), 1), (dict(nxt=FAKE + 4), 1),
    (dict(k=FAKE + 8), 1), (dict(path=FAKE + 2), 1), (dict(lens=FAKE + 4), 1), (dict(err=FAKE + 2), 1),
    (dict(batch=1 << 30, desc=(4, 8, 128, 64), lens=FAKE + (1 << 40)), 2),
])
def test_commit_refusals(lib, kw, status):
    assert commit(lib, **kw) == status


@pytest.mark.parametrize("out", ["path", "acc", "nxt", "lens"])
@pytest.mark.parametrize("src", ["draft", "target", "par", "cu", "sl", "bt"])
def test_commit_refuses_outputs_over_inputs(lib, out, src):
    """One byte in common is enough: the inputs are read by blocks that start at any time."""
    names = ["draft", "target", "par", "cu", "sl", "bt", "k", "v", "path", "acc", "nxt", "lens"]
    apart = {n: FAKE + (i << 20) for i, n in enumerate(names)}
    size = dict(draft=48, target=48, par=24, cu=12, sl=8, bt=24, path=24, acc=8, nxt=16, lens=8)
    step = 8 if out == "nxt" else 4
    low = size[src] - 1 - (size[src] - 1) % step     # the output begins in the input's last element
    assert commit(lib, **{**apart, out: apart[src] + low}) == 1
    assert commit(lib, **{**apart, src: apart[out] + size[out] - (8 if src in ("draft", "target") else 4)}) == 1


# ---- the binding --------------------------------------------------------------------------------
def rows(T=4, Hq=4, Hkv=2, B=2, P=3, dtype=torch.bfloat16):
    return dict(q=torch.zeros((T, Hq, 128), dtype=dtype), k_new=torch.zeros((T, Hkv, 128), dtype=dtype),
                v_new=torch.zeros((T, Hkv, 128), dtype=dtype), inv_freq=torch.zeros(64),
                positions=torch.zeros(B, dtype=torch.int32),
                block_table=torch.zeros((B, 3), dtype=torch.int32),
                q_out=torch.zeros((T, Hq, 128), dtype=dtype),
                k_cache=torch.zeros((P, Hkv, 64, 128), dtype=dtype),
                v_cache=torch.zeros((P, Hkv, 64, 128), dtype=dtype))


@pytest.mark.parametrize("kw", [
    dict(k_new=None), dict(v_new=None), dict(v_cache=None), dict(q=None), dict(q_out=None),
    dict(k_cache=None), dict(k_new=torch.zeros((4, 2, 128))),
    dict(k_new=torch.zeros((4, 2, 128), dtype=torch.float16)),
    dict(v_new=torch.zeros((3, 2, 128), dtype=torch.bfloat16)),
    dict(k_new=torch.zeros((4, 1, 128), dtype=torch.bfloat16)),
    dict(q_out=torch.zeros((4, 8, 128), dtype=torch.bfloat16)),
    dict(v_cache=torch.zeros((3, 2, 32, 128), dtype=torch.bfloat16)),
    dict(k_cache=torch.zeros((4, 2, 64, 128), dtype=torch.bfloat16)),
    dict(k_cache=torch.zeros((3, 2, 64, 128), dtype=torch.float16)),
    dict(inv_freq=torch.zeros(64, dtype=torch.float64)), dict(inv_freq=torch.zeros((64, 1))),
    dict(inv_freq=torch.zeros(128)[::2]), dict(inv_freq=torch.zeros(4)), dict(inv_freq=torch.zeros(72)),
    dict(positions=torch.zeros(2, dtype=torch.int64)), dict(positions=torch.zeros(3, dtype=torch.int32)),
    dict(block_table=torch.zeros(6, dtype=torch.int32)), dict(cu_tokens=torch.zeros(2, dtype=torch.int32)),
    dict(rope_positions=torch.zeros(3, dtype=torch.int32)),
    dict(rope_positions=torch.zeros(4, dtype=torch.int64)),
    dict(error_word=torch.zeros(3, dtype=torch.uint8)),
    dict(quantized=(torch.zeros((3, 2, 64), dtype=torch.uint8), torch.zeros((3, 2, 8704), dtype=torch.uint8))),
    dict(rot_scale=math.nan),
], ids=lambda kw: "-".join(kw))
def test_binding_refuses_appends(lib, kw):
    a = {**rows(), **kw}
    a = {n: OnGpu(x) if isinstance(x, torch.Tensor) else tuple(map(OnGpu, x)) if isinstance(x, tuple) else x
         for n, x in a.items()}
    with pytest.raises(ffd.FFDError):
        on_gpu_0(lambda: ffd.ffd_rope_append(
            a["q"], a["k_new"], a["v_new"], a["inv_freq"], a["positions"], a["block_table"], a["q_out"],
            a["k_cache"], a["v_cache"], cu_tokens=a.get("cu_tokens"),
            rope_positions=a.get("rope_positions"), rot_scale=a.get("rot_scale", 1.0),
            quantized=a.get("quantized"), error_word=a.get("error_word")))


def on_gpu_0(call):
    """The binding's call as if GPU 0 were there and current: what reaches the library is refused by it."""
    from sparse_quantized_attention_gb300 import ffd as binding

    class Fake:
        _cuda_getDevice = staticmethod(lambda: 0)
        _cuda_getCurrentRawStream = staticmethod(lambda dev: 0)

    before, binding._C = binding._C, Fake
    try:
        return call()
    finally:
        binding._C = before


def test_binding_refuses_cpu_tensors(lib):
    a = rows()
    with pytest.raises(ffd.FFDError):
        ffd.ffd_rope_append(a["q"], a["k_new"], a["v_new"], a["inv_freq"], a["positions"],
                            a["block_table"], a["q_out"], a["k_cache"], a["v_cache"])
    p = ffd.make_tree_params(2, 4, 2, 3, 3, max_q_len=2, num_splits=1)
    with pytest.raises(ffd.FFDError):
        ffd.ffd_tree_attention(p, a["q"], a["k_cache"], a["v_cache"], a["positions"], a["block_table"],
                               a["q_out"], torch.zeros(1 << 20))
    i, z = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ffd.FFDError):
        ffd.ffd_tree_commit(z, z, i, a["block_table"], a["k_cache"], a["v_cache"], i, i, z, i)


def test_binding_refuses_attention_tensors(lib):
    a = rows()
    p = ffd.make_tree_params(2, 4, 2, 3, 3, max_q_len=2, num_splits=1)
    z = dict(q=a["q"], k=a["k_cache"], v=a["v_cache"], sl=a["positions"], bt=a["block_table"],
             out=a["q_out"], ws=torch.zeros(64, dtype=torch.uint8), par=torch.zeros(4, dtype=torch.int32),
             cu=torch.zeros(3, dtype=torch.int32), keep=torch.zeros((2, 2, 3), dtype=torch.uint8),
             lse=torch.zeros((4, 4)))

    def call(**kw):
        x = {n: OnGpu(t) for n, t in {**z, **kw}.items()}
        with pytest.raises(ffd.FFDError) as e:
            ffd.ffd_tree_attention(p, x["q"], x["k"], x["v"], x["sl"], x["bt"], x["out"], x["ws"],
                                   parents=x["par"], cu_q=x["cu"], keep_in=x["keep"], lse=x["lse"])
        return str(e.value)

    assert "k and v" in call(k=z["k"].half())
    assert "k and v" in call(v=z["v"][:2])
    assert "k and v" in call(v=z["v"].transpose(0, 1))
    assert "k and v" in call(q=z["q"].half())
    assert "q and out" in call(out=z["out"][:2])
    assert "q's rows" in call(q=torch.zeros((4, 8, 128), dtype=torch.bfloat16)[:, :4])
    assert "int32" in call(sl=z["sl"].long())
    assert "int32" in call(par=z["par"][:3])
    assert "int32" in call(par=z["par"].long())
    assert "int32" in call(cu=z["cu"][:2])
    assert "keep_in" in call(keep=z["keep"].bool())
    assert "lse" in call(lse=z["lse"].half())
    assert "workspace" in call(ws=z["ws"][::2])


def test_binding_refuses_commit_tensors(lib):
    a = rows()
    i, z = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    base = dict(draft=torch.zeros(4, dtype=torch.int64), target=torch.zeros(4, dtype=torch.int64), sl=i,
                bt=a["block_table"], k=a["k_cache"], v=a["v_cache"], path=torch.zeros(4, dtype=torch.int32),
                acc=i, nxt=z, lens=i, par=torch.zeros(4, dtype=torch.int32),
                cu=torch.zeros(3, dtype=torch.int32))

    def call(**kw):
        x = {n: OnGpu(t) for n, t in {**base, **kw}.items()}
        with pytest.raises(ffd.FFDError) as e:
            on_gpu_0(lambda: ffd.ffd_tree_commit(
                x["draft"], x["target"], x["sl"], x["bt"], x["k"], x["v"], x["path"], x["acc"], x["nxt"],
                x["lens"], parents=x["par"], cu_nodes=x["cu"]))
        return str(e.value)

    assert "k_cache" in call(v=base["v"].float())
    assert "k_cache" in call(k=base["k"][:2])
    assert "int64 draft" in call(draft=base["path"])
    assert "int64 draft" in call(target=base["target"][:3])
    assert "int64 draft" in call(path=base["draft"])
    assert "int64 draft" in call(par=base["draft"])
    assert "int32 seq_lens" in call(acc=z)
    assert "int32 seq_lens" in call(nxt=i)
    assert "int32 seq_lens" in call(cu=base["cu"][:2])
    assert "INVALID_ARG" in call()      # new_lens is seq_lens
