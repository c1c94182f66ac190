"""What the two thread blocks of a wide tile hand to each other: a tile's rows are
split over them by row, its value columns by column, and neither may be ahead
of the other where it matters.  Each batch gives the two different work and
runs many times."""
import math

import pytest
import torch

from chunk_tail import with_fp16_tail
from chunk_utils import Batch

pytestmark = pytest.mark.gpu

KINDS = [("bf16", "bf16"), ("bf16", "fp8")]


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from indexer_top_sparse_c4_b200 import build, qsa
    build.build()
    return qsa


def _put_nan(b, r, p, col):
    """NaN as value `col` of request r's token p."""
    page, row = int(b.table[r, p // 64]), p % 64
    if b.kv_dt == "fp8":
        b.v.view(torch.uint8)[page, row, 0, col] = 0x7f
    else:
        b.v[page, row, 0, col] = math.nan


@pytest.mark.parametrize("late", [0, 1])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_nan_that_the_other_block_clears(q, q_dt, kv_dt, D, late):
    """16 heads and 16 tokens a request: tokens 0 to 7 are one block's rows, 8 to
    15 the other's.  In the last tile a key far above all others makes the rows
    of block `late` rescale their sums, so that it comes to the tile's values
    late; the NaN there lies in its columns, and rows of the other block see it."""
    lens = [(129 + i % 3, 16) for i in range(300)]     # enough tiles that none is split
    b = Batch(lens, 16, 1, D, q_dt, kv_dt, seed=40 + late)
    rows = torch.zeros(b.T, dtype=torch.bool, device="cuda")
    for t in range(b.T):
        rows[t] = (t % 16 >= 8) == bool(late)
    b.q[:, :, 0] = torch.where(rows, 64.0, 0.0)[:, None].to(b.q.dtype)
    b.k.view(torch.uint8 if kv_dt == "fp8" else b.k.dtype)[..., 0] = 0
    for r in range(b.B):
        b.k[int(b.table[r, 2]), 0, 0, 0] = torch.tensor(min(64.0 / b.k_scale, 448.0)).to(b.k.dtype)   # token 128
        if r % 4 == 0:
            continue                                    # its neighbours hold none
        _put_nan(b, r, int(b.kv_len[r]) - (1 if late == 0 else 12), 5 if late == 0 else D - 3)
    ref, ws, first = with_fp16_tail(b, b.reference()), b.workspace(q), None
    for _ in range(30):
        b.out.fill_(7.0)
        b.lse.fill_(7.0)
        b.run(q, workspace=ws)
        b.check(ref=ref)
        got = b.out.clone().view(torch.int16)
        assert first is None or torch.equal(first, got)
        first = got
    col = 5 if late == 0 else D - 3
    odd = torch.isnan(b.out[:, 0, col].float()).view(-1, 16)
    assert bool(odd[1, 15]) and not bool(odd[0].any()) and int(odd[1].sum()) == (1 if late == 0 else 12)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_full_items_before_nearly_empty_ones(q, q_dt, kv_dt, D):
    """16 tokens of 16 heads, every row of a tile, then a single token's long row,
    whose pieces leave most warps without a row and end anywhere: warps with
    nothing to do are an item ahead of the others."""
    lens = [x for i in range(40) for x in ((300 + 13 * i, 16), (3000 + 211 * i, 1))]
    b = Batch(lens, 16, 1, D, q_dt, kv_dt, seed=50)
    ref, ws, first = with_fp16_tail(b, b.reference()), b.workspace(q), None
    for _ in range(20):
        b.out.fill_(7.0)
        b.lse.fill_(7.0)
        b.run(q, workspace=ws)
        b.check(ref=ref)
        got = b.out.clone().view(torch.int16)
        assert first is None or torch.equal(first, got)
        first = got
