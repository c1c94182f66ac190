"""Block tables and slot maps, and the rotary cache write, against plain forms
(whole numbers exactly; floating values within their roundings)."""
import math

import numpy as np
import pytest
import torch

import chunk_utils as cu_

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from indexer_top_sparse_c4_b200 import build, qsa
    build.build()
    return qsa


def _plan(q, cached, new, T, num_pages=5000, width=40, n_free=None, table=None, seed=0, want=0, free=None):
    rng = np.random.default_rng(seed)
    B = len(cached)
    ids = rng.permutation(num_pages).astype(np.int32)
    if table is None:
        table = np.full((B + 2, width), -9, np.int32)
        at = 0
        for b, c in enumerate(cached):
            n = min(max(cu_.pages(max(c, 0)), 0), width)
            table[b, :n] = ids[at:at + n]
            at += n
        ids = ids[at:]
    free = ids[:n_free] if free is None else free
    i = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    dev = dict(cu=torch.full((B + 1,), -5, dtype=torch.int32, device="cuda"))
    out = {k: torch.full((n,), -5, dtype=torch.int32, device="cuda")
           for k, n in (("kv", B), ("req", T), ("pos", T), ("slot", T), ("taken", 1))}
    tab, status = i(table), torch.zeros(1, dtype=torch.int32, device="cuda")
    q.qsa_chunk_plan(i(cached), i(new), i(free), tab, num_pages, dev["cu"], out["kv"], out["req"], out["pos"],
                     out["slot"], out["taken"], dev_status=status)
    torch.cuda.synchronize()
    ref = table.copy()
    cu, kv, req, pos, slot, taken = cu_.plan_ref(cached, new, list(free), ref, num_pages, T)
    assert int(status.item()) == want
    assert dev["cu"].tolist() == cu and out["kv"].tolist() == kv and out["taken"].tolist() == [taken]
    assert out["req"].tolist() == req and out["pos"].tolist() == pos and out["slot"].tolist() == slot
    assert np.array_equal(tab.cpu().numpy(), ref)


@pytest.mark.parametrize("cached, new, T", [
    ([0], [1], 1), ([63], [1], 1), ([64], [1], 1), ([0], [64], 64), ([0], [65], 70), ([5, 0, 130], [3, 0, 200], 210),
    ([0, 0, 0], [0, 0, 0], 4), ([100, 64, 1], [0, 0, 0], 0), ([127] * 300, [1] * 300, 333),
])
def test_plan_small(q, cached, new, T):
    _plan(q, cached, new, T)


@pytest.mark.parametrize("B, T_pad, seed", [(1, 3, 0), (7, 0, 1), (257, 100, 2), (1031, 5, 3), (8192, 0, 4)])
def test_plan_random(q, B, T_pad, seed):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, 300, B)
    new = np.where(rng.random(B) < 0.3, 0, rng.integers(0, 40, B))
    _plan(q, cached.tolist(), new.tolist(), int(new.sum()) + T_pad, num_pages=60000, width=9, seed=seed)


def test_plan_bad_data(q):
    """Each is reported and served as the header says."""
    _plan(q, [-4, 10], [3, -2], 6, want=q.QSA_DEV_ROW_RANGE)                     # negative lengths
    _plan(q, [10, 20, 30], [5, 5, 5], 8, want=q.QSA_DEV_ROW_RANGE)               # tokens past T
    _plan(q, [100], [100], 100, width=2, want=q.QSA_DEV_ROW_RANGE)               # past the table's row
    _plan(q, [0, 0, 0], [64, 64, 64], 192, n_free=2, want=q.QSA_DEV_NO_PAGE)     # free list too short
    _plan(q, [0], [64], 64, n_free=0, want=q.QSA_DEV_NO_PAGE)
    _plan(q, [0, 0], [64, 64], 128, num_pages=100, free=np.array([100, 5], np.int32), want=q.QSA_DEV_BAD_PAGE)


# ---- rotary and cache write -------------------------------------------------------

def _rope(q, T, Hq, Hkv, D, rot, axes=1, inter=False, adj=False, x="bf16", kv="bf16", far=300000, seed=0, scale=1.0,
          pad=(), strided=True, in_place=False):
    g = torch.Generator(device="cpu").manual_seed(seed)
    X, half = cu_.TYPES[x], rot // 2
    if strided:
        qkv = torch.randn((T, (Hq + 2 * Hkv) * D + 16), generator=g).to(X).cuda()
        qx, kx, vx = (qkv[:, a:b].view(T, -1, D) for a, b in
                      ((0, Hq * D), (Hq * D, (Hq + Hkv) * D), ((Hq + Hkv) * D, (Hq + 2 * Hkv) * D)))
    else:
        qx, kx, vx = (torch.randn((T, h, D), generator=g).to(X).cuda() for h in (Hq, Hkv, Hkv))
    side = half // 3
    sec = {1: (half, 0, 0), 2: (half - side, side, 0), 3: (half - 2 * side, side, side)}[axes]
    pos = torch.randint(-5, far, (axes, T), generator=g, dtype=torch.int32).cuda()
    inv = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
    num_pages = T // 32 + 3
    slot = torch.randperm(num_pages * 64, generator=g)[:T].to(torch.int32)
    for i in pad:
        slot[i] = -1
    slot = slot.cuda()
    ks, vs = (0.011, 0.013) if kv == "fp8" else (1.0, 1.0)
    raw = torch.uint8 if kv == "fp8" else cu_.TYPES[kv]
    old = [torch.randint(0, 100, (num_pages, 64, Hkv, D), generator=g).to(raw).cuda() for _ in range(2)]
    kc, vc = (t.clone().view(cu_.TYPES[kv]) for t in old)
    q0, k0, v0 = qx.double(), kx.double(), vx.double()
    qo = qx if in_place else torch.full((T, Hq, D), 7.0, dtype=X, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.qsa_rope_write(qx, kx, vx, pos if axes > 1 else pos[0], inv, slot, qo, kc, vc, sections=sec,
                     interleaved_axes=inter, adjacent_pairs=adj, rot_scale=scale, k_scale=ks, v_scale=vs,
                     dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    axis = cu_.axis_ref(half, sec, inter)
    live = (slot >= 0)
    qr = cu_.rope_ref(q0, pos, inv, axis, adj, scale)
    kr = cu_.rope_ref(k0, pos, inv, axis, adj, scale)
    # A sine or cosine from a 32-bit fraction of a turn: the angle (at most pi)
    # is off by 2^-24 of itself twice (the fraction and its product with pi),
    # 2^-21.3, plus 2 units of the function and one of the scale: 2^-20.5 in
    # all; two products and their sum add 3 * 2^-24 of |a| + |b|.
    def tol(x0, ref, u):
        mag = torch.zeros_like(x0)
        i = torch.arange(half, device="cuda")
        i, j = (2 * i, 2 * i + 1) if adj else (i, i + half)
        m = (x0[..., i].abs() + x0[..., j].abs()) * abs(scale) * (2.0 ** -20.5 + 3 * 2.0 ** -24)
        mag[..., i], mag[..., j] = m, m
        return mag + u * (ref.abs() + mag)
    want = torch.where(live[:, None, None], qr, q0 if in_place else 7.0)
    t = torch.where(live[:, None, None], tol(q0, qr, torch.finfo(X).eps / 2), 0.0)
    assert bool(((qo.double() - want).abs() <= t).all())
    at = slot[live].long()
    for cache, was, ref, base, s in ((kc, old[0], kr, k0, ks), (vc, old[1], v0, None, vs)):
        got = cache.view(-1, Hkv, D)
        touched = torch.zeros(num_pages * 64, dtype=torch.bool, device="cuda")
        touched[at] = True
        assert torch.equal(got.view(raw)[~touched], was.view(-1, Hkv, D)[~touched])   # other rows stay
        y, r = got[at].double() * (s if kv == "fp8" else 1.0), ref[live]
        # an FP8 code: half a step of e4m3 (2^-4 of the value, 2^-10 of the scale
        # among the subnormals) and the quotient's own 2^-23
        u = 2.0 ** -4 + 2.0 ** -23 if kv == "fp8" else torch.finfo(cu_.TYPES[kv]).eps / 2
        if kv == "fp8":
            r = r.clamp(-448 * s, 448 * s)
        t = tol(base[live], r, u) if base is not None else u * r.abs()
        if base is None and kv == x:
            t = t * 0
        assert bool(((y - r).abs() <= t + (2.0 ** -10 * s * 1.001 if kv == "fp8" else 0.0)).all())


@pytest.mark.parametrize("x, kv", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"),
                                   ("f32", "fp8")])
@pytest.mark.parametrize("adj", [False, True])
@pytest.mark.parametrize("D, rot, Hq, Hkv", [(256, 64, 16, 2), (256, 256, 3, 1), (128, 128, 12, 1), (64, 16, 4, 4),
                                             (128, 48, 5, 5)])
def test_rope_types_and_pairs(q, D, rot, Hq, Hkv, adj, x, kv):
    _rope(q, 37, Hq, Hkv, D, rot, adj=adj, x=x, kv=kv, pad=(0, 5, 36))


@pytest.mark.parametrize("axes, inter", [(1, False), (1, True), (2, False), (2, True), (3, False), (3, True)])
@pytest.mark.parametrize("T", [1, 3, 1184, 1185, 2501])
def test_rope_axes_and_lengths(q, T, axes, inter):
    """One token to many: parts of a token's heads and whole tokens to a warp."""
    _rope(q, T, 4, 2, 128, 96, axes=axes, inter=inter, seed=T)


def test_rope_far_positions_keep_their_angles(q):
    """Positions near 2^31: a 32-bit angle would be off by whole turns."""
    _rope(q, 64, 2, 1, 64, 64, far=2 ** 31 - 1, x="f32", kv="f32")


def test_rope_scale_in_place_and_plain_rows(q):
    _rope(q, 21, 4, 1, 64, 32, scale=1.37, strided=False)
    for adj in (False, True):
        _rope(q, 1300, 6, 2, 128, 128, adj=adj, strided=False, in_place=True, pad=(3, 1299))


def test_rope_bad_slots_are_skipped(q):
    T, Hq, Hkv, D = 4, 2, 1, 64
    x = torch.ones((T, Hq, D), device="cuda")
    kv = torch.ones((T, Hkv, D), device="cuda")
    kc = torch.zeros((2, 64, Hkv, D), device="cuda")
    vc = torch.zeros_like(kc)
    qo = torch.full_like(x, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slot = torch.tensor([128, -2, 3, -1], dtype=torch.int32, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    q.qsa_rope_write(x, kv, kv, pos, torch.ones(32, device="cuda"), slot, qo, kc, vc, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == q.QSA_DEV_BAD_PAGE
    assert bool((qo[[0, 1, 3]] == 7).all()) and bool((qo[2] == 1).all())
    assert float(kc.sum()) == D and float(vc.sum()) == D and float(kc.view(-1, D)[3].sum()) == D


def test_rope_extreme_values_reach_the_fp8_cache(q):
    """Saturation, infinities and NaN: past +-448 codes to +-448, NaN to NaN."""
    D = 64
    v = torch.zeros((1, 1, D), device="cuda")
    v[0, 0, :6] = torch.tensor([1e9, -1e9, math.inf, -math.inf, math.nan, 448.0])
    kc = torch.zeros((1, 64, 1, D), dtype=torch.float8_e4m3fn, device="cuda")
    vc = torch.zeros_like(kc)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.qsa_rope_write(v.clone().nan_to_num(0, 0, 0), torch.zeros_like(v), v, z, torch.ones(32, device="cuda"), z,
                     torch.empty_like(v), kc, vc)
    got = vc[0, 0, 0, :6].float()
    assert got[:4].tolist() == [448, -448, 448, -448] and bool(got[4].isnan()) and float(got[5]) == 448


def test_rope_offsets_past_32_bits(q):
    """A cache of more than 2^32 values: the last page's rows."""
    Hkv, D = 16, 256
    num_pages = 2 ** 32 // (64 * Hkv * D) + 40
    kc = torch.zeros((num_pages, 64, Hkv, D), dtype=torch.float8_e4m3fn, device="cuda")
    vc = torch.zeros_like(kc)
    x = torch.randn((2, Hkv, D), device="cuda").to(torch.bfloat16)
    slot = torch.tensor([num_pages * 64 - 1, 5], dtype=torch.int32, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    q.qsa_rope_write(x, x, x, pos, torch.ones(32, device="cuda"), slot, torch.empty_like(x), kc, vc)
    want = x.float().to(torch.float8_e4m3fn).view(torch.uint8)
    for c in (kc, vc):
        assert torch.equal(c[-1, 63].view(torch.uint8), want[0]) and torch.equal(c[0, 5].view(torch.uint8), want[1])
        assert int(c.view(torch.uint8).view(num_pages, -1)[1:-1].max()) == 0
