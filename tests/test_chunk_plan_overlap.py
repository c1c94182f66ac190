"""qsa_chunk_plan's inputs are read by every thread block while others write its
outputs, so a call whose outputs lie over its inputs is refused (on the host,
before anything is launched)."""
import ctypes

import pytest

B, T, N_FREE, ROWS, WIDTH = 5, 40, 12, 6, 8
SIZES = dict(n_cached=B, n_new=B, free_pages=N_FREE, page_table=B * WIDTH, cu_new=B + 1, kv_len=B, q_req=T, q_pos=T,
             slot=T, n_taken=1)
INPUTS = ("n_cached", "n_new", "free_pages")


@pytest.fixture(scope="module")
def L():
    from indexer_top_sparse_c4_b200 import build, qsa
    build.build()
    return qsa.lib()


def _addresses():
    """One buffer after the other, 4 bytes a value."""
    at, out = 0x10000, {}
    for name, n in SIZES.items():
        out[name] = at
        at += 4 * n
    return out


def _call(L, a, B=B, T=-1):
    p = {k: ctypes.c_void_p(v) for k, v in a.items()}
    return L.qsa_chunk_plan(p["n_cached"], p["n_new"], B, p["free_pages"], N_FREE, p["page_table"], ROWS, WIDTH, 100,
                            40 if T < 0 else T, p["cu_new"], p["kv_len"], p["q_req"], p["q_pos"], p["slot"],
                            p["n_taken"], None, None)


@pytest.mark.parametrize("src", INPUTS)
@pytest.mark.parametrize("dst", [n for n in SIZES if n not in INPUTS])
@pytest.mark.parametrize("edge", ["first", "last"])
def test_outputs_over_inputs_are_refused(L, src, dst, edge):
    """The output's last value on the input's first, and the other way round."""
    a = _addresses()
    far = 0x40000000
    a[src] = far
    a[dst] = far - 4 * (SIZES[dst] - 1) if edge == "first" else far + 4 * (SIZES[src] - 1)
    assert _call(L, a) == 1
    assert "overlap" in L.qsa_last_error_string().decode()


def test_lengths_in_place_are_refused(L):
    a = _addresses()
    a["kv_len"] = a["n_cached"]
    assert _call(L, a) == 1 and "kv_len" in L.qsa_last_error_string().decode()
