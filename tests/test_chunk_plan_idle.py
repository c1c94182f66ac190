"""An idle step (no requests) on the host: what qsa_chunk_plan and qsa_chunk_attn
need and what they refuse."""
import ctypes

import pytest

OK = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def L():
    from indexer_top_sparse_c4_b200 import build, qsa
    build.build()
    return qsa.lib()


@pytest.mark.parametrize("cu, taken, T, q", [(None, OK, 0, None), (OK, None, 0, None), (None, None, 4, OK), (OK, OK, 4, None)])
def test_idle_step_needs_its_outputs(L, cu, taken, T, q):
    """The counts of an idle step are results like any other: a caller that asks
    for one of them, or for padded rows, gives all that are written."""
    assert L.qsa_chunk_plan(None, None, 0, None, 0, None, 0, 4, 8, T, cu, None, q, q, q, taken, None, None) == 1
    assert "null" in L.qsa_last_error_string().decode()


def test_requests_still_need_theirs(L):
    assert L.qsa_chunk_plan(None, OK, 1, None, 0, OK, 1, 4, 8, 4, OK, OK, OK, OK, OK, OK, None, None) == 1
    assert L.qsa_chunk_plan(OK, OK, 1, None, 0, None, 1, 4, 8, 4, OK, OK, OK, OK, OK, OK, None, None) == 1
    assert L.qsa_chunk_plan(OK, OK, 1, None, 0, OK, 0, 4, 8, 4, OK, OK, OK, OK, OK, OK, None, None) == 1


def _attn(L, B, rows, T=4):
    return L.qsa_chunk_attn(OK, 1, OK, OK, 1, 1.0, 1.0, 8, OK, rows, 4, OK, OK, B, T, 16, 2, 256, 0.0, OK, None, OK,
                            1 << 40, None, None)


def test_idle_attention_takes_a_table_without_rows(L):
    """The table of a batch of no requests, [0, pages], as the plan takes it."""
    assert _attn(L, 0, 0) == 0 and _attn(L, 0, 2) == 0 and _attn(L, 0, 0, T=0) == 0
    assert _attn(L, 1, 0) == 1 and _attn(L, 0, -1) == 1
