"""Block tables of steps at the ends of the range: idle steps without requests."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from indexer_top_sparse_c4_b200 import build, qsa
    build.build()
    return qsa


def _ints(*shape, fill=-5):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rows", [0, 2])
@pytest.mark.parametrize("T", [0, 1, 77, 3000])
def test_an_idle_step_has_results_of_its_own(q, T, rows):
    """No request at all: no token, no page taken, and padding behind."""
    cu, kv, taken, table, status = _ints(1), _ints(0), _ints(1), _ints(rows, 4), _ints(1, fill=0)
    req, pos, slot = (_ints(T) for _ in range(3))
    q.qsa_chunk_plan(_ints(0), _ints(0), _ints(9), table, 16, cu, kv, req, pos, slot, taken, dev_status=status)
    assert cu.tolist() == [0] and taken.tolist() == [0] and int(status.item()) == 0
    for t in (req, pos, slot):
        assert bool((t == -1).all())
    assert bool((table == -5).all())
