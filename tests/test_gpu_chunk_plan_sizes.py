"""Block tables of steps at the ends of the range: idle steps without requests,
and batches around the size where the kernel's shared memory has to be asked
for."""
import os
import subprocess
import sys

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


def test_buffers_side_by_side(q):
    """All arrays slices of one buffer, each behind the other: nothing overlaps,
    an exhausted free list of no pages inside another array neither."""
    B, T = 3, 9
    sizes = dict(old=B, new=B, table=B * 2, cu=B + 1, kv=B, req=T, pos=T, slot=T, taken=1)
    buf, at, v = _ints(sum(sizes.values())), 0, {}
    for name, n in sizes.items():
        v[name] = buf[at:at + n]
        at += n
    v["old"].copy_(torch.tensor([3, 64, 0], dtype=torch.int32))
    v["new"].copy_(torch.tensor([5, 0, 0], dtype=torch.int32))
    table = v["table"].view(B, 2)
    table[:, 0] = torch.arange(B, dtype=torch.int32, device="cuda")
    q.qsa_chunk_plan(v["old"], v["new"], v["slot"][4:4], table, 8, v["cu"], v["kv"], v["req"], v["pos"], v["slot"],
                     v["taken"])
    assert v["cu"].tolist() == [0, 5, 5, 5] and v["kv"].tolist() == [8, 64, 0] and v["taken"].tolist() == [0]
    assert v["pos"].tolist() == [3, 4, 5, 6, 7, -1, -1, -1, -1] == v["slot"].tolist()


def test_a_free_list_in_a_spare_row_of_the_table(q):
    """Rows past the batch's are not written and may hold anything."""
    table = _ints(3, 8)
    table[2] = torch.arange(10, 18, dtype=torch.int32, device="cuda")
    cu, kv, taken, (req, pos, slot) = _ints(3), _ints(2), _ints(1), (_ints(70) for _ in range(3))
    q.qsa_chunk_plan(_ints(2, fill=0), torch.tensor([64, 6], dtype=torch.int32, device="cuda"), table[2], table, 20, cu, kv,
                     req, pos, slot, taken)
    assert taken.tolist() == [2] and table[:2, 0].tolist() == [10, 11] and table[2].tolist() == list(range(10, 18))
    assert slot.tolist() == list(range(640, 704)) + list(range(704, 710))


SIZES = """
import torch
from indexer_top_sparse_c4_b200 import qsa
i = lambda n, fill=-5: torch.full((n,), fill, dtype=torch.int32, device="cuda")
for B in (6135, 6136, 6143, 6144, 8192):
    cu, kv, taken, status = i(B + 1), i(B), i(1), i(1, 0)
    req, pos, slot = i(B), i(B), i(B)
    free = torch.arange(B, dtype=torch.int32, device="cuda")
    qsa.qsa_chunk_plan(i(B, 0), i(B, 1), free, i(B).view(B, 1), B, cu, kv, req, pos, slot, taken, dev_status=status)
    want = torch.arange(B, device="cuda")
    assert int(status) == 0 and int(taken) == B and int(cu[B]) == B
    assert torch.equal(req.long(), want) and torch.equal(slot.long(), want * 64) and bool((pos == 0).all())
print("served")
"""


def test_every_batch_size_in_a_process_of_its_own(q):
    """Sizes in ascending order, before any larger one has raised a limit."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SIZES], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "served" in r.stdout, r.stderr[-2000:]
