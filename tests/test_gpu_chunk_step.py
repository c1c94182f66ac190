"""The dense chunk step as a serving loop runs it: tables and slots, rotary and
cache write, attention -- prompts, then single tokens, then drafts -- against a
plain form in 64 bits that keeps every request's rotated keys and values."""
import math

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


class Loop:
    """Buffers of a loop of at most T tokens a step, and its plain form."""

    def __init__(self, q, B, T, Hq, Hkv, D, x, kv, axes, seed):
        self.q, self.B, self.T, self.Hq, self.Hkv, self.D, self.axes = q, B, T, Hq, Hkv, D, axes
        self.X, self.KV = cu_.TYPES[x], cu_.TYPES[kv]
        self.g = torch.Generator().manual_seed(seed)
        ints = dict(dtype=torch.int32, device="cuda")
        self.num_pages, width = 70, 12
        self.free = torch.randperm(self.num_pages, generator=self.g).to(torch.int32).cuda()
        self.table = torch.full((B, width), -1, **ints)
        self.k_scale, self.v_scale = (0.02, 0.0125) if kv == "fp8" else (1.0, 1.0)
        raw = torch.uint8 if kv == "fp8" else self.KV
        bad = 0x7f if kv == "fp8" else math.nan           # rows nobody wrote must not matter
        self.kc = torch.full((self.num_pages, 64, Hkv, D), bad, dtype=raw, device="cuda").view(self.KV)
        self.vc = self.kc.clone()
        self.n_cached, self.n_new = torch.zeros(B, **ints), torch.zeros(B, **ints)
        self.cu, self.kv_len = torch.zeros(B + 1, **ints), torch.zeros(B, **ints)
        self.req, self.pos, self.slot = (torch.zeros(T, **ints) for _ in range(3))
        self.pos3 = torch.zeros((axes, T), **ints)
        self.taken, self.status = torch.zeros(1, **ints), torch.zeros(1, **ints)
        self.qkv = torch.zeros((T, (Hq + 2 * Hkv) * D), dtype=self.X, device="cuda")
        self.qr, self.out = (torch.zeros((T, Hq, D), dtype=self.X, device="cuda") for _ in range(2))
        self.lse = torch.zeros((T, Hq), device="cuda")
        half = D // 2
        self.inv_freq = (1e4 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        self.sec = [half] if axes == 1 else [half - 2 * (half // 3), half // 3, half // 3]
        n = q.qsa_chunk_attn_workspace_size(T, B, Hq, Hkv, D, self.KV)
        self.ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
        self.keys = [torch.zeros((0, Hkv, D), dtype=torch.float64, device="cuda") for _ in range(B)]
        self.vals = [k.clone() for k in self.keys]
        self.at = 0                                       # pages taken from the free list so far

    def calls(self):
        q, H, K, D, T = self.q, self.Hq, self.Hkv, self.D, self.T
        q.qsa_chunk_plan(self.n_cached, self.n_new, self.free_now, self.table, self.num_pages, self.cu, self.kv_len,
                         self.req, self.pos, self.slot, self.taken, dev_status=self.status)
        self.pos3.copy_(self.pos.expand(self.axes, T))    # text: every axis runs with the token
        x = self.qkv
        q.qsa_rope_write(x[:, :H * D].view(T, H, D), x[:, H * D:(H + K) * D].view(T, K, D),
                         x[:, (H + K) * D:].view(T, K, D), self.pos3, self.inv_freq, self.slot, self.qr, self.kc, self.vc,
                         sections=self.sec, k_scale=self.k_scale, v_scale=self.v_scale, dev_status=self.status)
        q.qsa_chunk_attn(self.qr, self.kc, self.vc, self.table, self.cu, self.kv_len, self.out, workspace=self.ws,
                         k_scale=self.k_scale, v_scale=self.v_scale, lse=self.lse, dev_status=self.status)

    def step(self, news, run=None):
        """One step of `news` new tokens a request; checks all it produced."""
        self.free_now = self.free[self.at:] if run is None else self.free_now
        self.n_cached.copy_(torch.tensor([len(k) for k in self.keys], dtype=torch.int32))
        self.n_new.copy_(torch.tensor(news, dtype=torch.int32))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=self.g))
        self.out.fill_(7.0)
        self.lse.fill_(7.0)
        (run or self.calls)()
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        used = sum(news)
        H, K, D = self.Hq, self.Hkv, self.D
        x = self.qkv[:used].double()
        qd, kd, vd = (x[:, a * D:(a + n) * D].reshape(used, n, D) for a, n in ((0, H), (H, K), (H + K, K)))
        pos = torch.cat([len(k) + torch.arange(n, device="cuda") for k, n in zip(self.keys, news)])
        assert torch.equal(self.pos[:used].long(), pos) and bool((self.pos[used:] == -1).all())
        axis = cu_.axis_ref(D // 2, [*self.sec, 0, 0][:3], False)
        p3 = pos.expand(self.axes, used)
        qd = cu_.rope_ref(qd, p3, self.inv_freq, axis, False, 1.0)
        kd = cu_.rope_ref(kd, p3, self.inv_freq, axis, False, 1.0)
        # the cache holds values of its type; those are what attention reads
        kk = self.kc.view(-1, K, D)[self.slot[:used].long()].double() * self.k_scale
        vv = self.vc.view(-1, K, D)[self.slot[:used].long()].double() * self.v_scale
        step = {torch.float32: 2.0 ** -20, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}[self.KV]
        for got, want, s in ((kk, kd, self.k_scale), (vv, vd, self.v_scale)):
            assert bool(((got - want).abs() <= 1.01 * step * want.abs() + 2.0 ** -10 * s + 2.0 ** -19).all())
        t, G = 0, H // K
        u = torch.finfo(self.X).eps / 2
        u_p = 0.0 if self.X == torch.float32 else 2.0 ** -8 if self.KV == torch.bfloat16 else 2.0 ** -11
        for b, n in enumerate(news):
            rows = slice(t, t + n)
            self.keys[b] = torch.cat([self.keys[b], kk[rows]])
            self.vals[b] = torch.cat([self.vals[b], vv[rows]])
            t += n
            L = len(self.keys[b])
            if n == 0:
                continue
            qh = self.qr[rows].double().view(n, K, G, D)   # the rotated queries as rounded, checked below
            want = qd[rows].view(n, K, G, D)
            assert bool(((qh - want).abs() <= u * want.abs() + 2.0 ** -18).all())
            s = torch.einsum("nkgd,lkd->nkgl", qh, self.keys[b]) / math.sqrt(D)
            mag = torch.einsum("nkgd,lkd->nkgl", qh.abs(), self.keys[b].abs()).amax(-1) / math.sqrt(D)
            hide = torch.arange(L, device="cuda") > (L - n + torch.arange(n, device="cuda"))[:, None]
            s = s.masked_fill(hide[:, None, None], -math.inf)
            z = torch.logsumexp(s, -1)
            pr = torch.exp(s - z[..., None])
            o = torch.einsum("nkgl,lkd->nkgd", pr, self.vals[b])
            A = torch.einsum("nkgl,lkd->nkgd", pr, self.vals[b].abs())
            # a logit: D + 8 roundings of FP32 of its terms and the exponential's 2^-22;
            # the sums (L + 16) 2^-24; a probability's rounding u_p; the output's own
            rel = u_p + 2 * ((D + 8) * 2.0 ** -24 * mag + 2.0 ** -22) + 2 * (L + 16) * 2.0 ** -24
            tol = rel[..., None] * A + u * (o.abs() + rel[..., None] * A) + 1e-30
            assert bool(((self.out[rows].double().view(n, K, G, D) - o).abs() <= tol).all())
            assert bool(((self.lse[rows].double().view(n, K, G) - z).abs() <= rel + 2.0 ** -22 * (z.abs() + 1)).all())
        assert bool((self.out[used:] == 7).all()) and bool((self.lse[used:] == 7).all())
        self.at += int(self.taken.item())


@pytest.mark.parametrize("x, kv, axes, Hq, Hkv, D", [("bf16", "bf16", 1, 16, 2, 256), ("bf16", "fp8", 3, 12, 1, 128),
                                                     ("bf16", "fp8", 1, 16, 2, 256), ("bf16", "bf16", 3, 4, 4, 64),
                                                     ("f32", "f32", 3, 4, 1, 64)])
def test_prompts_then_tokens_then_drafts(q, x, kv, axes, Hq, Hkv, D):
    loop = Loop(q, 4, 300, Hq, Hkv, D, x, kv, axes, seed=D + axes)
    loop.step([100, 1, 0, 64])       # prompts, one of them later
    loop.step([57, 130, 3, 64])      # their second chunks
    loop.step([1, 1, 1, 1])
    loop.step([4, 2, 3, 1])
    loop.step([0, 70, 1, 2])         # a chunk among single tokens
    loop.step([1, 1, 0, 1])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_captured_step_serves_every_batch(q, kv):
    """One captured graph of the three calls, padded, replayed for steps of
    different lengths: everything that changes is read on the device."""
    loop = Loop(q, 4, 160, 16, 2, 128, "bf16", kv, 1, seed=5)
    loop.free_now = torch.full((loop.num_pages,), -1, dtype=torch.int32, device="cuda")
    loop.n_new.zero_()
    loop.calls()
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        loop.calls()

    def run():
        rest = loop.free[loop.at:]
        loop.free_now[:rest.numel()].copy_(rest)
        g.replay()
    for news in ([60, 1, 30, 64], [1, 1, 1, 1], [2, 100, 3, 1], [1, 0, 1, 1], [0, 0, 0, 0], [4, 4, 4, 4]):
        loop.step(news, run=run)


def test_bound_calls(q):
    """The rotary and attention calls bound once, called again on refilled
    buffers; scales and sections as numpy and torch scalars."""
    import numpy as np
    b = cu_.Batch([(200, 2), (0, 33)], 8, 2, 128, "bf16", "fp8", seed=7)
    ws = b.workspace(q)
    b.k_scale, b.v_scale = np.float32(b.k_scale), torch.tensor(b.v_scale)
    go = q.bind(b.run, q, workspace=ws)
    torch.cuda.synchronize()
    assert bool((b.out == 7).all())          # binding ran nothing
    b.k_scale, b.v_scale = float(b.k_scale), float(b.v_scale)
    for _ in range(2):
        b.q.copy_(torch.randn(b.q.shape, device="cuda"))
        go()
        b.check()
    x = torch.zeros((3, 4, 64), device="cuda")
    kc, vc = (torch.zeros((1, 64, 4, 64), device="cuda") for _ in range(2))
    pos = torch.zeros((3, 3), dtype=torch.int32, device="cuda")
    slot = torch.arange(3, dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    go = q.bind(q.qsa_rope_write, x, x, x, pos, torch.ones(32, device="cuda"), slot, out, kc, vc,
                sections=np.array([12, 10, 10]), rot_scale=np.float64(2.0))
    x.fill_(3.0)
    go()
    torch.cuda.synchronize()
    assert bool((out == 6).all()) and bool((kc.view(-1, 4, 64)[:3] == 6).all()) and bool((vc.view(-1, 4, 64)[:3] == 3).all())
