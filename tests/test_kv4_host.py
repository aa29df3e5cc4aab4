"""Refusals of the 4-bit cache's entries (no GPU needed): bad arguments come back as a status, or as
an FFDError from the binding, before anything is enqueued."""
import ctypes
import math

import pytest
import torch

import sparse_quantized_attention_gb300 as ffd
from sparse_quantized_attention_gb300 import _build

FAKE = 0x10000  # never dereferenced: every call here fails validation first


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ffd.lib()


def test_exports_and_version(lib):
    raw = ctypes.CDLL(_build.LIB)
    for name in ("ffd_kv4_write", "ffd_kv4_read", "ffd_kv4_workspace_size", "ffd_kv4_attention"):
        assert hasattr(raw, name)
    assert ffd.ffd_version() == 310


def rows_call(lib, read, desc=(4, 2, 128, 64), dtype=0, batch=2, mb=3, total=6, ks=256, vs=256,
              **kw):
    a = dict(k=FAKE, v=FAKE, cu=FAKE, pos=FAKE, bt=FAKE, k4=FAKE, v4=FAKE)
    a.update(kw)
    d = ctypes.byref(ffd.CacheDesc(*desc)) if desc else None
    if read:
        return lib.ffd_kv4_read(d, dtype, batch, mb, total, a["cu"], a["pos"], a["bt"], a["k4"],
                                a["v4"], a["k"], ks, a["v"], vs, None, None)
    return lib.ffd_kv4_write(d, dtype, batch, mb, total, a["k"], ks, a["v"], vs, a["cu"], a["pos"],
                             a["bt"], a["k4"], a["v4"], None, None)


@pytest.mark.parametrize("read", [False, True], ids=["write", "read"])
@pytest.mark.parametrize("kw,status", [
    (dict(desc=None), 1),
    (dict(desc=(0, 2, 128, 64)), 1),
    (dict(desc=(4, 0, 128, 64)), 1),
    (dict(desc=(4, 2, 64, 64)), 2),
    (dict(desc=(4, 2, 128, 32)), 2),
    (dict(dtype=2), 1),
    (dict(dtype=-1), 1),
    (dict(batch=0), 1),
    (dict(mb=0), 1),
    (dict(mb=1 << 26), 2),
    (dict(total=-1), 1),
    (dict(cu=None, total=5), 1),       # rows not shared out evenly
    (dict(ks=255), 1),
    (dict(ks=260), 1),
    (dict(vs=128), 1),
    (dict(k=FAKE + 8), 1),
    (dict(v=FAKE + 2), 1),
    (dict(k4=FAKE + 8), 1),
    (dict(v4=None), 1),
    (dict(cu=FAKE + 2), 1),
    (dict(pos=None), 1),
    (dict(bt=None), 1),
    (dict(k=None, v=None), 1),
    (dict(desc=(4, 1 << 20, 128, 64), ks=1 << 27, vs=1 << 27, total=1 << 30), 2),
])
def test_rows_refusals(lib, read, kw, status):
    assert rows_call(lib, read, **kw) == status


def test_write_wants_both_tensors(lib):
    assert rows_call(lib, False, k=None) == 1
    assert rows_call(lib, False, v=None) == 1


def test_no_rows_is_no_work(lib):
    assert rows_call(lib, False, total=0) == 0
    assert rows_call(lib, True, total=0) == 0


def params(**kw):
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, num_pages=10, max_blocks_per_seq=5,
                max_q_len=3, total_q=6, num_splits=2)
    base.update(kw)
    return ffd.make_kv4_params(base.pop("batch"), base.pop("num_q_heads"),
                               base.pop("num_kv_heads"), base.pop("num_pages"),
                               base.pop("max_blocks_per_seq"), **base)


def attend(lib, p, ws_bytes=1 << 40, **kw):
    a = dict(q=FAKE, k4=FAKE, v4=FAKE, sl=FAKE, cu=FAKE, bt=FAKE, keep=None, out=FAKE, lse=None,
             ws=FAKE)
    a.update(kw)
    return lib.ffd_kv4_attention(ctypes.byref(p) if p else None, *[a[k] for k in (
        "q", "k4", "v4", "sl", "cu", "bt", "keep", "out", "lse", "ws")], ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 1),
    (dict(num_q_heads=7), 1),
    (dict(num_q_heads=18), 2),          # G = 9
    (dict(num_pages=0), 1),
    (dict(max_blocks_per_seq=0), 1),
    (dict(max_blocks_per_seq=1 << 26), 2),
    (dict(max_q_len=0), 1),
    (dict(total_q=0), 1),
    (dict(window=-1), 1),
    (dict(num_splits=-1), 1),
    (dict(wait_limit_us=-1), 1),
    (dict(sm_scale=0.0), 1),
    (dict(sm_scale=-1.0), 1),
    (dict(sm_scale=math.nan), 1),
    (dict(sm_scale=math.inf), 1),
    (dict(q_stride=8), 1),
    (dict(q_stride=1028), 1),
    (dict(batch=40000), 2),
    (dict(num_pages=1 << 30), 2),
    (dict(max_q_len=1 << 27), 2),
    (dict(max_blocks_per_seq=1 << 24, batch=200, total_q=600), 2),
])
def test_attention_refuses_params(lib, kw, status):
    p = params(**kw)
    assert attend(lib, p) == status
    assert ffd.ffd_kv4_workspace_size(p) == 0


def test_attention_refuses_shapes_and_pointers(lib):
    p = params()
    need = ffd.ffd_kv4_workspace_size(p)
    assert need > 0 and need % 256 == 0
    for field, value, status in (("head_dim", 64, 2), ("page_size", 16, 2), ("dtype", 3, 1)):
        bad = params()
        setattr(bad, field, value)
        assert attend(lib, bad) == status
    assert attend(lib, None) == 1
    for key in ("q", "k4", "v4", "sl", "bt", "out", "ws"):
        assert attend(lib, p, **{key: None}) == 1, key
    for key, off in (("q", 8), ("k4", 4), ("v4", 8), ("out", 2), ("ws", 16), ("cu", 2), ("sl", 1),
                     ("lse", 2)):
        assert attend(lib, p, **{key: FAKE + off}) == 1, key
    assert attend(lib, p, ws_bytes=need - 1) == 3
    # without offsets every sequence has max_q_len rows
    assert attend(lib, params(total_q=5), cu=None) == 1


def test_attention_refuses_out_over_q(lib):
    p = params()                        # q and out are 6 rows of 8 heads: 12288 bytes each
    assert attend(lib, p) == 1
    assert attend(lib, p, out=FAKE + 12288 - 16) == 1
    assert attend(lib, p, q=FAKE + 12288 - 16) == 1
    p = params(q_stride=2048)           # out between the first and the second row of q
    assert attend(lib, p, out=FAKE + 2048) == 1


def test_binding_refuses_tensors(lib):
    """CPU tensors and wrong shapes or types never reach a kernel."""
    bt = torch.zeros((2, 3), dtype=torch.int32)
    pos = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros((2, 2, 128), dtype=torch.bfloat16)
    cache = ffd.alloc_kv4_cache(4, 2, device="cpu")
    with pytest.raises(ffd.FFDError):
        ffd.ffd_kv4_write(x, x, pos, bt, cache)
    with pytest.raises(ffd.FFDError):
        ffd.ffd_kv4_read(cache, pos, bt, x, None)
    p = params(max_q_len=1, total_q=2)
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ffd.FFDError):
        ffd.ffd_kv4_attention(p, q, cache, pos, bt, q.clone(), torch.zeros(1 << 20))
    def stride(y, heads=2):
        return ffd.ffd._row_stride(y, y.shape[0], heads, torch.bfloat16)

    assert stride(x) == 256 and stride(x, heads=1) is None and stride(x.float()) is None
    assert stride(x.transpose(1, 2), heads=128) is None
    wide = torch.zeros((2, 600), dtype=torch.bfloat16)
    assert stride(wide[:, 8:264].unflatten(1, (2, 128))) == 600
    assert stride(wide[:, :512:2].unflatten(1, (2, 128))) is None
    assert stride(wide[:1, 8:264].unflatten(1, (2, 128))) == 256  # one row: any distance
    with pytest.raises(ffd.FFDError):
        ffd.ffd_kv4_write(None, x, pos, bt, cache)
    with pytest.raises(ffd.FFDError):
        ffd.ffd_kv4_read(cache, pos, bt, None, None)


class OnGpu:
    """A CPU tensor that says it is on GPU 0: what the checks after the devices' see."""

    def __init__(self, t):
        self.t = t

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_refuses_shapes_and_types(lib):
    P, Hkv, B, T = 4, 2, 2, 3
    z = dict(k4=torch.zeros((P, Hkv, 5120), dtype=torch.uint8),
             v4=torch.zeros((P, Hkv, 5120), dtype=torch.uint8),
             pos=torch.zeros(B, dtype=torch.int32), bt=torch.zeros((B, 3), dtype=torch.int32),
             k=torch.zeros((T, Hkv, 128), dtype=torch.float16),
             v=torch.zeros((T, Hkv, 128), dtype=torch.float16),
             cu=torch.zeros(B + 1, dtype=torch.int32))

    def rows(**kw):
        a = {n: OnGpu(t) for n, t in {**z, **kw}.items()}
        with pytest.raises(ffd.FFDError) as e:
            ffd.ffd_kv4_read((a["k4"], a["v4"]), a["pos"], a["bt"], a["k"], a["v"],
                             cu_tokens=a["cu"])
        return str(e.value)

    assert "the cache" in rows(k4=z["k4"][:, :, :64])
    assert "the cache" in rows(v4=z["v4"][:2])
    assert "the cache" in rows(v4=z["v4"].float())
    assert "the cache" in rows(k4=z["k4"].transpose(0, 1))
    assert "int32" in rows(pos=z["pos"].long())
    assert "int32" in rows(pos=torch.zeros(3, dtype=torch.int32))
    assert "int32" in rows(bt=torch.zeros((B, 6), dtype=torch.int32)[:, ::2])
    assert "int32" in rows(bt=torch.zeros(6, dtype=torch.int32))
    assert "int32" in rows(cu=torch.zeros(B, dtype=torch.int32))
    assert "rows" in rows(k=z["k"].float())
    assert "rows" in rows(v=z["v"].bfloat16())
    assert "rows" in rows(v=z["v"][:2])
    assert "rows" in rows(k=torch.zeros((T, Hkv, 256), dtype=torch.float16)[..., ::2])

    Hq = 8
    p = ffd.make_kv4_params(B, Hq, Hkv, P, 3, total_q=T, max_q_len=2, num_splits=1)
    y = dict(z, q=torch.zeros((T, Hq, 128), dtype=torch.bfloat16),
             out=torch.zeros((T, Hq, 128), dtype=torch.bfloat16),
             sl=torch.zeros(B, dtype=torch.int32), ws=torch.zeros(64, dtype=torch.uint8),
             keep=torch.zeros((B, Hkv, 3), dtype=torch.uint8), lse=torch.zeros((T, Hq)))

    def attend(**kw):
        a = {n: OnGpu(t) for n, t in {**y, **kw}.items()}
        with pytest.raises(ffd.FFDError) as e:
            ffd.ffd_kv4_attention(p, a["q"], (a["k4"], a["v4"]), a["sl"], a["bt"], a["out"],
                                  a["ws"], cu_q=a["cu"], keep_in=a["keep"], lse=a["lse"])
        return str(e.value)

    assert "the cache" in attend(k4=torch.zeros((P + 1, Hkv, 5120), dtype=torch.uint8))
    assert "q and out" in attend(q=y["q"].half())
    assert "q and out" in attend(out=y["out"][:2])
    assert "q and out" in attend(out=torch.zeros((T, Hq, 256), dtype=torch.bfloat16)[..., :128])
    assert "q's rows" in attend(q=torch.zeros((T, 2 * Hq, 128), dtype=torch.bfloat16)[:, :Hq])
    assert "q's rows" in attend(q=torch.zeros((T, Hq, 256), dtype=torch.bfloat16)[..., ::2])
    assert "int32" in attend(sl=torch.zeros(3, dtype=torch.int32))
    assert "int32" in attend(bt=torch.zeros((B, 4), dtype=torch.int32))
    assert "int32" in attend(cu=torch.zeros(B + 1))
    assert "keep_in" in attend(keep=y["keep"].bool())
    assert "lse" in attend(lse=y["lse"].double())
    assert "workspace" in attend(ws=torch.zeros(64, dtype=torch.uint8)[::2])
