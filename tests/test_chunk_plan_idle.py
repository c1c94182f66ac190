"""An idle step of qsa_chunk_plan on the host: what it needs and what it refuses."""
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
