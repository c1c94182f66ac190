"""Attention of a chunk of new tokens over the paged cache, against the plain
form in 64 bits; rows behind the last token of a request, pages nobody owns and
unused page-table entries hold NaN and ids out of range throughout."""
import math

import pytest
import torch

from chunk_utils import Batch

pytestmark = pytest.mark.gpu

KINDS = [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32")]


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from indexer_top_sparse_c4_b200 import build, qsa
    build.build()
    return qsa


def _run(q, *args, **kw):
    b = Batch(*args, **kw)
    b.run(q)
    b.check()
    return b


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
@pytest.mark.parametrize("Hq, Hkv, D", [(16, 2, 256), (24, 2, 256), (12, 1, 128), (6, 1, 128), (3, 1, 256), (4, 1, 64),
                                        (8, 8, 64), (16, 1, 128), (5, 5, 128)])
def test_mixed_batch(q, Hq, Hkv, D, q_dt, kv_dt):
    """Single tokens, drafts, whole prompts and chunks of them, an empty request."""
    lens = [(0, 1), (63, 1), (64, 1), (500, 3), (0, 0), (0, 130), (77, 45), (1000, 1), (126, 2)]
    _run(q, lens, Hq, Hkv, D, q_dt, kv_dt, seed=D + Hq, pad=3)


@pytest.mark.parametrize("q_dt, kv_dt", KINDS + [("f32", "bf16"), ("f32", "fp8"), ("bf16", "f32")])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_dtype_pairs(q, D, q_dt, kv_dt):
    _run(q, [(200, 5), (0, 70)], 4, 2, D, q_dt, kv_dt)


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
@pytest.mark.parametrize("kv", [1, 2, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 385])
def test_single_token_lengths(q, kv, q_dt, kv_dt):
    _run(q, [(kv - 1, 1)], 8, 1, 128, q_dt, kv_dt, seed=kv)


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 127, 128, 129, 300])
def test_prompt_lengths(q, n, q_dt, kv_dt):
    _run(q, [(0, n)], 8, 1, 256, q_dt, kv_dt, seed=n)


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_long_rows_are_split_and_merged(q, q_dt, kv_dt):
    """Few rows over many keys: every CTA takes a piece of a row."""
    _run(q, [(20000, 1), (37, 1), (9000, 2)], 16, 2, 256, q_dt, kv_dt)
    _run(q, [(30011, 1)], 3, 1, 128, q_dt, kv_dt)


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_many_tiles_are_not_split(q, q_dt, kv_dt):
    """Enough query tiles for whole tiles per CTA, in several requests."""
    n = 1500 if q_dt == "bf16" else 700
    _run(q, [(300, n), (0, 400), (5, 1), (0, n // 2)], 16, 2, 128, q_dt, kv_dt, pad=2)


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_many_requests(q, q_dt, kv_dt):
    """The largest batch, most of it short."""
    lens = [((i * 7) % 90, (i * 5) % 3) for i in range(1024)]
    _run(q, lens, 4, 2, 64, q_dt, kv_dt)


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_sharp_and_growing_logits(q, q_dt, kv_dt):
    """Logits of tens: the running maximum moves often and by much."""
    b = Batch([(700, 40)], 8, 2, 128, q_dt, kv_dt, k_mean=0.0, seed=3)
    b.q.mul_(8)
    b.run(q)
    b.check()
    b.run(q, sm_scale=0.31)
    b.check(sm_scale=0.31)


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_query_rows_of_very_different_size(q, q_dt, kv_dt):
    """Rows from 2^-60 to 2^40: an FP8 cache's product takes the query in FP16."""
    b = Batch([(100, 30)], 4, 1, 128, q_dt, kv_dt, seed=4)
    e = torch.linspace(-60, 3, b.T, device="cuda").round()
    b.q.copy_((b.q.float() * torch.exp2(e)[:, None, None]).to(b.q.dtype))
    b.q[3] = 0
    b.run(q)
    b.check()
    b.q[:, :, :64] *= 2.0 ** -12           # within a row, too
    b.run(q)
    b.check()


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_rows_without_keys(q, q_dt, kv_dt):
    """kv_len 0, or shorter than the new tokens: zeros and -inf."""
    b = Batch([(0, 5), (3, 20), (0, 1)], 8, 1, 128, q_dt, kv_dt, seed=5)
    b.kv_len[0] = 0
    b.kv_len[1] = 11         # positions -9 .. 10
    b.run(q)
    b.check()
    assert float(b.out[:5].abs().max()) == 0 and bool(torch.isneginf(b.lse[:5]).all())
    assert bool(torch.isneginf(b.lse[5:14]).all()) and bool(torch.isfinite(b.lse[14:25]).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_values_a_row_does_not_see(q, q_dt, kv_dt, bad):
    """NaN or infinity in a new token's value (and key) reaches the rows at and
    behind it only."""
    if kv_dt == "fp8" and not math.isnan(bad):
        pytest.skip("e4m3 has no infinities")
    b = Batch([(130, 90), (0, 40)], 8, 2, 128, q_dt, kv_dt, seed=6)
    p = 130 + 37
    page, row = int(b.table[0, p // 64]), p % 64
    if kv_dt == "fp8":
        b.v.view(torch.uint8)[page, row, 1, 5] = 0x7f
    else:
        b.v[page, row, 1, 5] = bad
    b.run(q)
    b.check()
    p = 130 + 60
    page, row = int(b.table[0, p // 64]), p % 64
    if kv_dt == "fp8":
        b.k.view(torch.uint8)[page, row, 0, 5] = 0xff
    else:
        b.k[page, row, 0, 5] = math.nan
    b.run(q)
    b.check()
    assert bool(torch.isfinite(b.out[:37].float()).all())


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_bad_pages_are_skipped_and_reported(q, q_dt, kv_dt):
    b = Batch([(300, 20), (0, 100)], 8, 2, 128, q_dt, kv_dt, seed=7)
    b.table[0, 1] = b.num_pages
    b.table[0, 3] = -1
    b.table[1, 0] = 2 ** 31 - 1
    b.run(q)
    torch.cuda.synchronize()
    bits = int(b.status.item())
    assert bits == q.QSA_DEV_BAD_PAGE
    b.table[0, 1] = b.table[0, 3] = b.table[1, 0] = 0      # the reference leaves them out
    b.check(status=bits, skip=((0, 1), (0, 3), (1, 0)))


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_lengths_past_the_table_are_reported(q, q_dt, kv_dt):
    b = Batch([(300, 4)], 8, 2, 128, q_dt, kv_dt, seed=8)
    b.table = b.table[:, :3].contiguous()                   # 192 of 304 tokens
    b.run(q)
    torch.cuda.synchronize()
    assert int(b.status.item()) == q.QSA_DEV_ROW_RANGE
    b.status.zero_()
    ok = Batch([(188, 4)], 8, 2, 128, q_dt, kv_dt, seed=8)
    ok.q, ok.k, ok.v, ok.table = b.q, b.k, b.v, b.table
    out, lse, tol, ltol = ok.reference()
    # every row sees all 192 tokens: the last row of the shorter request
    out, lse = out[3:].expand(4, -1, -1).clone(), lse
    assert b.out.shape == out.shape
    ok.out, ok.lse = b.out[3:].clone(), b.lse[3:].clone()
    ok.check(ref=(out[3:], lse[3:], tol[3:], ltol[3:]))


def test_corrupt_offsets_are_reported(q):
    b = Batch([(100, 4), (100, 4)], 8, 2, 128, seed=9)
    b.cu.copy_(torch.tensor([0, 9, 5], dtype=torch.int32))
    b.run(q)
    torch.cuda.synchronize()
    assert int(b.status.item()) == q.QSA_DEV_ROW_RANGE
    b.cu.copy_(torch.tensor([-3, 2 ** 30, -2 ** 31], dtype=torch.int32))
    b.status.zero_()
    b.run(q)
    torch.cuda.synchronize()
    assert int(b.status.item()) == q.QSA_DEV_ROW_RANGE


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_results_do_not_change(q, q_dt, kv_dt):
    """The same call twice, and over another workspace's leftovers: bit-equal;
    lse may be left out; captured and replayed with other lengths."""
    b = Batch([(5000, 1), (333, 7), (0, 64)], 16, 2, 128, q_dt, kv_dt, seed=10, pad=1)
    b.run(q)
    first, flse = b.out.clone(), b.lse.clone()
    b.out.fill_(7.0)
    b.lse.fill_(7.0)
    ws = torch.zeros_like(b.workspace(q))
    b.run(q, workspace=ws)
    assert torch.equal(first, b.out) and torch.equal(flse, b.lse)
    b.out.fill_(7.0)
    q.qsa_chunk_attn(b.q, b.k, b.v, b.table, b.cu, b.kv_len, b.out, workspace=ws, k_scale=b.k_scale, v_scale=b.v_scale)
    assert torch.equal(first, b.out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        b.run(q, workspace=ws)
    torch.cuda.synchronize()
    for kv in ([5001, 340, 64], [17, 8, 64], [4000, 7, 70]):
        b.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        b.out.fill_(7.0)
        b.lse.fill_(7.0)
        b.status.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        if kv[2] > 64:            # two pages, the second not the request's own: reported
            assert int(b.status.item()) == q.QSA_DEV_BAD_PAGE
            continue
        b.check()


def test_two_streams_with_their_own_workspaces(q):
    a = Batch([(9000, 1)], 16, 2, 256, "bf16", "fp8", seed=11)
    c = Batch([(0, 700)], 16, 2, 256, "bf16", "bf16", seed=12)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    w1, w2 = a.workspace(q), c.workspace(q)
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(q, workspace=w1, stream=s1)
        c.run(q, workspace=w2, stream=s2)
    a.check()
    c.check()


@pytest.mark.parametrize("kv_dt", ["bf16", "fp8"])
def test_offsets_past_32_bits(q, kv_dt):
    """A cache of more than 2^32 values whose last pages are the request's."""
    from chunk_utils import TYPES
    Hkv, D = 16, 256
    b = Batch([(200, 2)], 16, Hkv, D, "bf16", kv_dt, seed=13)
    n = 2 ** 32 // (64 * Hkv * D) + 64
    for name in ("k", "v"):
        small = getattr(b, name)
        big = torch.zeros((n, 64, Hkv, D), dtype=TYPES[kv_dt], device="cuda")
        big[-b.num_pages:].copy_(small)
        setattr(b, name, big)
    used = 4
    b.table[0, :used] += n - b.num_pages
    b.num_pages = n
    b.run(q)
    b.check()


def test_chunk_attention_equals_the_dense_rows_of_the_sparse_path(q):
    """The same chunk through dense token lists and the sparse prefill kernel."""
    b = Batch([(60, 130)], 16, 2, 256, "bf16", "bf16", seed=14)
    b.run(q)
    b.check()
    pos = torch.arange(60, 190, dtype=torch.int32, device="cuda")
    tok = torch.empty((130, 256), dtype=torch.int32, device="cuda")
    n_tok = torch.empty(130, dtype=torch.int32, device="cuda")
    q.qsa_dense_select(pos, 1 << 20, tok, n_tok)
    out = torch.empty_like(b.out)
    req = torch.zeros(130, dtype=torch.int32, device="cuda")
    q.qsa_sparse_attn_prefill(b.q, b.k, b.v, b.table, tok, n_tok, out, q_req=req)
    # both round the probabilities (2^-8) and the output (2^-8) to bf16
    _, _, tol, _ = b.reference()
    assert bool(((out.double() - b.out.double()).abs() <= 2 * tol).all())


# ---- requests of a few rows: the kernel of decode steps and drafts -----------------

DRAFTS = [(0, 1), (1, 2), (15, 1), (14, 2), (16, 1), (63, 2), (200, 2), (0, 0), (1000, 1), (30, 2), (5, 1), (4095, 2)]


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
@pytest.mark.parametrize("Hq, Hkv, D", [(16, 2, 256), (8, 1, 128), (24, 2, 256), (16, 1, 64), (3, 1, 256), (6, 2, 128),
                                        (4, 4, 64), (1, 1, 128), (5, 5, 256)])
def test_drafts(q, Hq, Hkv, D, q_dt, kv_dt):
    """One and two tokens a request, padded: every tile height and head group."""
    _run(q, DRAFTS, Hq, Hkv, D, q_dt, kv_dt, seed=20 + D + Hq, pad=2)
    _run(q, [(n, 1) for n, _ in DRAFTS], Hq, Hkv, D, q_dt, kv_dt, seed=21 + D + Hq)


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_a_chunk_among_single_tokens(q, q_dt, kv_dt):
    """Many single tokens and one long chunk: the chunk's tiles are narrow ones."""
    _run(q, [(i * 13, 1) for i in range(150)] + [(70, 151)], 8, 2, 128, q_dt, kv_dt, seed=22)


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
@pytest.mark.parametrize("D", [64, 256])
def test_drafts_hidden_values_and_bad_pages(q, D, q_dt, kv_dt):
    """NaN in the last token's value reaches that token's row only; a NaN key
    likewise; pages out of range are skipped and reported."""
    b = Batch([(300, 2), (77, 2), (500, 1)], 4, 1, D, q_dt, kv_dt, seed=23)
    for r, what in ((0, b.v), (1, b.k)):
        p = int(b.kv_len[r]) - 1
        page, row = int(b.table[r, p // 64]), p % 64
        if kv_dt == "fp8":
            what.view(torch.uint8)[page, row, 0, 3] = 0x7f
        else:
            what[page, row, 0, 3] = math.nan if r else math.inf
    b.run(q)
    b.check()
    assert bool(torch.isfinite(b.out[[0, 2, 4]].float()).all())
    good = b.table.clone()
    b.table[0, 2], b.table[2, 0], b.table[2, 7] = -1, b.num_pages, 2 ** 31 - 1
    b.run(q)
    torch.cuda.synchronize()
    assert int(b.status.item()) == q.QSA_DEV_BAD_PAGE
    b.table.copy_(good)
    b.check(status=q.QSA_DEV_BAD_PAGE, skip=((0, 2), (2, 0), (2, 7)))


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_drafts_sharp_logits_and_row_sizes(q, q_dt, kv_dt):
    b = Batch([(3000, 2), (60, 2), (9, 1)], 8, 2, 128, q_dt, kv_dt, seed=24)
    b.q.mul_(8)
    b.run(q)
    b.check()
    b.q.copy_((b.q.float() * torch.exp2(torch.tensor([-60., 3., -20., 0., 9.], device="cuda"))[:, None, None]).to(b.q.dtype))
    b.q[3] = 0
    b.run(q)
    b.check()


@pytest.mark.parametrize("q_dt, kv_dt", KINDS)
def test_one_key_above_a_long_tail(q, q_dt, kv_dt):
    """One token far above 60,000 equal ones whose probabilities are tiny each
    and a good part of the output together."""
    b = Batch([(60000, 1)], 2, 1, 128, q_dt, kv_dt, seed=25)
    b.q.zero_()
    b.q[:, :, 0] = 8.0
    top = float(1.0 / b.k_scale) if kv_dt == "fp8" else 1.0
    b.k.view(torch.uint8).zero_() if kv_dt == "fp8" else b.k.zero_()
    page, row = int(b.table[0, 100]), 17
    b.k[page, row, 0, 0] = torch.tensor(min(15.6 * top, 448.0)).to(b.k.dtype)   # about 11 above the rest
    b.v.copy_((b.v.float().abs()).to(b.v.dtype))
    b.run(q)
    b.check()


@pytest.mark.parametrize("q_dt, kv_dt", KINDS[:2])
def test_drafts_captured_and_repeated(q, q_dt, kv_dt):
    b = Batch([(5000, 1), (333, 2), (0, 1)], 16, 2, 256, q_dt, kv_dt, seed=26, pad=1)
    ws = b.workspace(q)
    b.run(q, workspace=ws)
    b.check()
    first, flse = b.out.clone(), b.lse.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        b.run(q, workspace=ws)
    for kv in ([5001, 335, 1], [17, 2, 1], [3000, 200, 0]):
        b.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        b.out.fill_(7.0)
        b.lse.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        b.check()
        if kv[0] == 5001:
            assert torch.equal(first, b.out) and torch.equal(flse, b.lse)


# ---- wide tiles: several items a worker, whole tiles, long rows in many parts -------

@pytest.mark.parametrize("q_dt, kv_dt", KINDS[:2])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_more_tiles_than_are_split(q, D, q_dt, kv_dt):
    """Four tiles a worker and more: every tile is one worker's, in rounds."""
    _run(q, [(i % 70, 17) for i in range(170)], 16, 1, D, q_dt, kv_dt, seed=30 + D, pad=1)


@pytest.mark.parametrize("q_dt, kv_dt", KINDS[:2])
def test_more_tiles_than_the_table_holds(q, q_dt, kv_dt):
    _run(q, [(i % 9, 17) for i in range(530)], 16, 1, 64, q_dt, kv_dt, seed=31)
    _run(q, [(40, 1000)] + [(i % 130, 1) for i in range(1000)], 4, 1, 64, q_dt, kv_dt, seed=32)


@pytest.mark.parametrize("q_dt, kv_dt", KINDS[:2])
@pytest.mark.parametrize("Hq, Hkv, D", [(16, 2, 256), (12, 1, 128), (8, 8, 64)])
def test_wide_tiles_over_long_rows(q, Hq, Hkv, D, q_dt, kv_dt):
    """A tile that every worker has a part of, beside short ones."""
    _run(q, [(30011, 33)], Hq, Hkv, D, q_dt, kv_dt, seed=33)
    _run(q, [(7000, 40), (3, 19), (129, 64), (0, 1), (4000, 21)], Hq, Hkv, D, q_dt, kv_dt, seed=34, pad=4)


@pytest.mark.parametrize("q_dt, kv_dt", KINDS[:2])
def test_hidden_values_over_several_items(q, q_dt, kv_dt):
    """Non-finite values in the last pages of some requests, in either half of a
    head: each reaches the rows at and behind it, no other item."""
    lens = [(100 + 7 * i, 24) for i in range(160)]
    b = Batch(lens, 16, 2, 128, q_dt, kv_dt, seed=35)
    for r, d, back in ((3, 5, 4), (3, 100, 1), (50, 127, 20), (159, 64, 24)):
        p = int(b.kv_len[r]) - back
        page, row = int(b.table[r, p // 64]), p % 64
        if kv_dt == "fp8":
            b.v.view(torch.uint8)[page, row, r % 2, d] = 0xff
        else:
            b.v[page, row, r % 2, d] = math.inf if r % 2 else math.nan
    b.run(q)
    b.check()
    odd = (~torch.isfinite(b.out.float())).any(-1).any(-1).nonzero().flatten().tolist()
    want = [24 * r + 24 - back + i for r, back in ((3, 4), (50, 20), (159, 24)) for i in range(back)]
    assert odd == sorted(want)


@pytest.mark.parametrize("kv_dt", ["bf16", "fp8"])
def test_two_graphs_in_turn(q, kv_dt):
    """Two captured calls of different shapes, each with its workspace, replayed
    in turn on one stream."""
    a = Batch([(2000, 1), (90, 1)], 16, 2, 256, "bf16", kv_dt, seed=36)
    c = Batch([(500, 70), (0, 33)], 16, 2, 256, "bf16", kv_dt, seed=37)
    graphs = []
    for b in (a, c):
        ws = b.workspace(q)
        b.run(q, workspace=ws)
        torch.cuda.synchronize()
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            b.run(q, workspace=ws)
        b.out.fill_(7.0)
        b.lse.fill_(7.0)
        graphs.append((g, ws))
    torch.cuda.synchronize()
    for _ in range(4):
        for g, _ws in graphs:
            g.replay()
    a.check()
    c.check()
