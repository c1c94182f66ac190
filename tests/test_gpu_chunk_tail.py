"""Probabilities far below a row's largest over an FP8 cache: FP16 subnormals,
which are rounded by up to 2^-32 of the largest whatever their own size."""
import pytest
import torch

from chunk_tail import with_fp16_tail
from chunk_utils import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from indexer_top_sparse_c4_b200 import build, qsa
    build.build()
    return qsa


@pytest.mark.parametrize("below", [18, 20, 21, 22, 24, 26, 28, 30, 31, 32, 33, 40])
@pytest.mark.parametrize("lens, Hq, Hkv", [([(6000, 1), (30, 1)], 2, 1), ([(900, 2), (70, 1)], 16, 2), ([(2000, 40)], 8, 1)])
def test_a_tail_below_the_normal_range(q, lens, Hq, Hkv, below):
    """One token 2^`below` above all others, whose value is zero in half of the
    columns: there the tail alone makes the output."""
    D = 128
    b = Batch(lens, Hq, Hkv, D, "bf16", "fp8", seed=60 + below)
    top = 448 * b.k_scale / D ** 0.5 * 1.4426950408889634      # base-2 logit of the highest code on a query of 1
    b.q.zero_()
    b.q[:, :, 0] = round(below / top)
    for r in range(b.B):
        ids = b.table[r, :-(-int(b.kv_len[r]) // 64)].long()
        codes = b.k.view(torch.uint8)[ids]
        codes[..., 0] = torch.where(codes[..., 0] == 0x7f, codes[..., 0], 0)
        b.k.view(torch.uint8)[ids] = codes
        page, row = int(b.table[r, 0]), 11
        b.k[page, row, :, 0] = torch.tensor(448.0).to(b.k.dtype)
        b.v.view(torch.uint8)[page, row, :, : D // 2] = 0
    b.run(q)
    b.check(ref=with_fp16_tail(b, b.reference()))
