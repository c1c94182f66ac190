"""The dense chunk step's calls on the host: what they refuse, before anything
is launched (no GPU needed)."""
import ctypes

import pytest
import torch

NULL = None
OK = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10004)


@pytest.fixture(scope="module")
def L():
    from indexer_top_sparse_c4_b200 import build, qsa
    build.build()
    return qsa.lib()


def _err(L):
    return L.qsa_last_error_string().decode()


def _plan(L, B=2, T=8, n_free=4, pt_rows=2, pt_stride=4, num_pages=16, ptr=OK, free=OK):
    return L.qsa_chunk_plan(ptr, ptr, B, free, n_free, ptr, pt_rows, pt_stride, num_pages, T, ptr, ptr, ptr, ptr, ptr,
                            ptr, NULL, NULL)


@pytest.mark.parametrize("kw, status, text", [
    (dict(B=-1), 1, ">= 0"), (dict(T=-1), 1, ">= 0"), (dict(n_free=-1), 1, ">= 0"),
    (dict(B=8193, pt_rows=9000), 2, "8192 requests"), (dict(T=(1 << 20) + 1), 2, "tokens per call"),
    (dict(pt_rows=1), 1, "page-table rows"), (dict(pt_stride=0), 1, "pt_stride"),
    (dict(pt_stride=(1 << 24) + 1), 2, "pt_stride"), (dict(num_pages=1 << 25), 2, "num_pages"),
    (dict(num_pages=0), 1, "num_pages"), (dict(ptr=NULL), 1, "null"), (dict(free=NULL), 1, "free_pages"),
])
def test_plan_refusals(L, kw, status, text):
    assert _plan(L, **kw) == status and text in _err(L)


def _rope(L, T=4, Hq=4, Hkv=2, D=128, rot=64, axes=1, sec=(32, 0, 0), inter=0, x_dt=1, kv_dt=1, q=OK, ptr=OK,
          qs=512, ks=256, vs=256, pos_stride=4, num_pages=8, scale=1.0, rot_scale=1.0):
    return L.qsa_rope_write(q, qs, ptr, ks, ptr, vs, x_dt, ptr, axes, pos_stride, *sec, inter, 0, ptr, rot, rot_scale,
                            ptr, T, Hq, Hkv, D, ptr, ptr, ptr, kv_dt, scale, scale, num_pages, NULL, NULL)


@pytest.mark.parametrize("kw, status, text", [
    (dict(T=-1), 1, "T must"), (dict(T=(1 << 20) + 1), 2, "tokens per call"), (dict(Hq=0), 1, "Hq"),
    (dict(D=96), 2, "head dim"), (dict(rot=24, sec=(12, 0, 0)), 1, "rot_dim"), (dict(rot=144, sec=(72, 0, 0)), 1, "rot_dim"),
    (dict(rot=0, sec=(0, 0, 0)), 1, "rot_dim"), (dict(axes=0), 1, "axes"), (dict(axes=4), 1, "axes"),
    (dict(sec=(31, 0, 0)), 1, "add up"), (dict(sec=(33, -1, 0), axes=2), 1, "add up"),
    (dict(sec=(16, 16, 0)), 1, "without an axis"), (dict(sec=(16, 8, 8), axes=2), 1, "without an axis"),
    (dict(sec=(16, 16, 0), axes=2, inter=1), 1, "interleaved"), (dict(sec=(21, 0, 11), axes=3, inter=1), 1, "interleaved"),
    (dict(axes=2, sec=(16, 16, 0), pos_stride=3), 1, "pos_stride"), (dict(x_dt=2), 1, "dtype"), (dict(kv_dt=7), 1, "dtype"),
    (dict(kv_dt=2, scale=0.0), 1, "scales"), (dict(kv_dt=2, scale=float("nan")), 1, "scales"),
    (dict(rot_scale=float("inf")), 1, "rot_scale"), (dict(qs=511), 1, "strides"), (dict(qs=516), 2, "multiples of 8"),
    (dict(vs=260), 2, "multiples of 8"), (dict(num_pages=1 << 25), 2, "num_pages"), (dict(num_pages=0), 1, "num_pages"),
    (dict(q=NULL), 1, "null"), (dict(q=ODD), 1, "aligned"),
])
def test_rope_refusals(L, kw, status, text):
    assert _rope(L, **kw) == status and text in _err(L)


def _attn(L, T=4, B=2, Hq=16, Hkv=2, D=256, q_dt=1, kv_dt=1, ptr=OK, q=OK, pt_rows=2, pt_stride=4, num_pages=8,
          scale=1.0, sm=0.0, ws=OK, ws_bytes=1 << 40):
    return L.qsa_chunk_attn(q, q_dt, ptr, ptr, kv_dt, scale, scale, num_pages, ptr, pt_rows, pt_stride, ptr, ptr, B, T,
                            Hq, Hkv, D, sm, ptr, NULL, ws, ws_bytes, NULL, NULL)


@pytest.mark.parametrize("kw, status, text", [
    (dict(T=-1), 1, ">= 0"), (dict(B=-1), 1, ">= 0"), (dict(T=(1 << 20) + 1), 2, "tokens per call"),
    (dict(B=1025, pt_rows=2000), 2, "requests per call"), (dict(Hq=6, Hkv=4), 1, "Hq % Hkv"),
    (dict(Hq=17, Hkv=1), 2, "16 query heads"), (dict(D=96), 2, "head dim"), (dict(B=3), 1, "page-table rows"),
    (dict(num_pages=1 << 25), 2, "num_pages"), (dict(pt_stride=0), 1, "pt_stride"),
    (dict(pt_stride=(1 << 24) + 1), 2, "pt_stride"), (dict(q_dt=2), 1, "q dtype"), (dict(kv_dt=5), 1, "KV dtype"),
    (dict(pt_stride=(1 << 20) + 1), 2, "pt_stride"),
    (dict(kv_dt=2, scale=-1.0), 1, "FP8"), (dict(sm=float("nan")), 1, "sm_scale"), (dict(ptr=NULL), 1, "null"),
    (dict(q=ODD), 1, "aligned"), (dict(ws=NULL), 3, "workspace"), (dict(ws_bytes=1024), 3, "workspace"),
    (dict(ws=ODD), 3, "workspace"),
])
def test_attention_refusals(L, kw, status, text):
    assert _attn(L, **kw) == status and text in _err(L)


def test_empty_calls_launch_nothing(L):
    assert _plan(L, B=0, T=0, ptr=NULL, free=NULL) == 0
    assert _rope(L, T=0, q=NULL, ptr=NULL) == 0
    assert _attn(L, T=0, ptr=NULL, q=NULL, ws=NULL) == 0
    assert _attn(L, B=0, ptr=NULL, q=NULL, ws=NULL) == 0
    assert L.qsa_chunk_plan_workspace_size(100, 8) == 0
    assert L.qsa_rope_write_workspace_size(100, 16, 2, 256) == 0
    assert L.qsa_chunk_attn_workspace_size(8192, 1, 24, 2, 256, 1) > 0


def test_binding_refuses_what_the_library_cannot_see():
    """Shapes, dtypes and strides that a pointer does not tell."""
    from indexer_top_sparse_c4_b200 import qsa
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    plan = dict(n_cached=i(2), n_new=i(2), free_pages=i(4), page_table=i(2, 4), num_pages=8, cu_new=i(3), kv_len=i(2),
                q_req=i(5), q_pos=i(5), slot=i(5), n_taken=i(1))
    with pytest.raises(ValueError, match="shapes"):
        qsa.qsa_chunk_plan(**{**plan, "cu_new": i(2)})
    with pytest.raises(TypeError, match="int32"):
        qsa.qsa_chunk_plan(**{**plan, "slot": torch.zeros(5, dtype=torch.int64)})

    def rope(**kw):
        a = dict(q=torch.zeros(5, 4, 64), k=torch.zeros(5, 2, 64), v=torch.zeros(5, 2, 64), pos=i(5),
                 inv_freq=torch.zeros(32), slot=i(5), q_out=torch.zeros(5, 4, 64), k_pages=torch.zeros(2, 64, 2, 64),
                 v_pages=torch.zeros(2, 64, 2, 64))
        return qsa.qsa_rope_write(**{**a, **kw})
    with pytest.raises(ValueError, match="contiguous"):
        rope(q=torch.zeros(5, 64, 4).transpose(1, 2))
    with pytest.raises(ValueError, match="sections"):
        rope(pos=i(3, 5))
    with pytest.raises(TypeError, match="one dtype"):
        rope(k=torch.zeros(5, 2, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="k_pages"):
        rope(k_pages=torch.zeros(2, 32, 2, 64))
    with pytest.raises(ValueError, match="pos"):
        rope(pos=i(4))

    def attn(**kw):
        a = dict(q=torch.zeros(5, 4, 64), k_pages=torch.zeros(2, 64, 2, 64), v_pages=torch.zeros(2, 64, 2, 64),
                 page_table=i(2, 4), cu_new=i(3), kv_len=i(2), out=torch.zeros(5, 4, 64))
        return qsa.qsa_chunk_attn(**{**a, **kw})
    with pytest.raises(ValueError, match="out"):
        attn(out=torch.zeros(5, 4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="lse"):
        attn(lse=torch.zeros(5, 3))
    with pytest.raises(ValueError, match="shapes"):
        attn(cu_new=i(2))


def test_binding_refuses_tensors_in_host_memory():
    """A kernel must never be given a host address."""
    from indexer_top_sparse_c4_b200 import qsa
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        qsa.qsa_chunk_plan(i(2), i(2), i(4), i(2, 4), 8, i(3), i(2), i(5), i(5), i(5), i(1))
    with pytest.raises(ValueError, match="CUDA"):
        qsa.qsa_rope_write(z(5, 4, 64), z(5, 2, 64), z(5, 2, 64), i(5), z(32), i(5), z(5, 4, 64), z(2, 64, 2, 64),
                           z(2, 64, 2, 64))
    with pytest.raises(ValueError, match="CUDA"):
        qsa.qsa_chunk_attn(z(5, 4, 64), z(2, 64, 2, 64), z(2, 64, 2, 64), i(2, 4), i(3), i(2), z(5, 4, 64))
