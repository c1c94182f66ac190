"""Plain 64-bit forms of the dense chunk step's operators, and the batches its
tests run on."""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE = 64
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


def pages(n):
    return -(-n // PAGE)


# ---- plan -----------------------------------------------------------------------

def plan_ref(cached, new, free, table, num_pages, T):
    """Lists in, lists out; table is changed in place."""
    cu, kv, req, pos, slot = [0], [], [-1] * T, [-1] * T, [-1] * T
    taken = t = 0
    width = table.shape[1]
    for b, (c, n) in enumerate(zip(cached, new)):
        c, n = max(c, 0), max(n, 0)
        n = min(n, T - t)
        kv.append(c + n)
        for i in range(min(pages(c), width), min(pages(c + n), width)):
            table[b, i] = free[taken] if taken < len(free) else -1
            taken += 1
        for i in range(n):
            req[t], pos[t] = b, c + i
            lp = pos[t] // PAGE
            page = table[b, lp] if lp < width else -1
            if 0 <= page < num_pages:
                slot[t] = page * PAGE + pos[t] % PAGE
            t += 1
        cu.append(t)
    return cu, kv, req, pos, slot, min(taken, len(free))


# ---- rotary ----------------------------------------------------------------------

def axis_ref(half, sec, interleaved):
    if not interleaved:
        return [0] * sec[0] + [1] * sec[1] + [2] * sec[2]
    axis = [0] * half
    for a in (1, 2):
        for n in range(sec[a]):
            axis[3 * n + a] = a
    return axis


def rope_ref(x, pos, inv_freq, axis, adjacent, scale):
    """x [T, H, D] float64, pos [A, T], inv_freq [half]: rotated, in 64 bits."""
    half = len(axis)
    p = pos.double()[torch.tensor(axis, device=x.device)]            # [half, T]
    a = (p * inv_freq.double()[:, None]).T[:, None]                  # [T, 1, half]
    c, s = torch.cos(a) * scale, torch.sin(a) * scale
    y = x.clone()
    i = torch.arange(half, device=x.device)
    i, j = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


# ---- attention --------------------------------------------------------------------

class Batch:
    """A batch of requests over a permuted paged cache.  Rows behind a request's
    last token, pages nobody owns and unused page-table entries hold values
    that must never show: NaN and page ids out of range."""

    def __init__(self, lens, Hq, Hkv, D, q_dt="bf16", kv_dt="bf16", seed=0, pad=0, device="cuda", spare=3, k_mean=0.0):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.lens, self.Hq, self.Hkv, self.D, self.B = lens, Hq, Hkv, D, len(lens)
        n_new = [n for _, n in lens]
        self.used = sum(n_new)
        self.T = self.used + pad
        kv = [c + n for c, n in lens]
        total = sum(pages(x) for x in kv)
        self.num_pages = total + spare
        width = max([pages(x) for x in kv] + [1]) + 2
        ids = torch.randperm(self.num_pages, generator=g)
        table = torch.full((self.B, width), 10 ** 9, dtype=torch.int32)
        table[:, -1] = -7
        self.k_scale, self.v_scale = (0.0123, 0.0317) if kv_dt == "fp8" else (1.0, 1.0)
        shape = (self.num_pages, PAGE, Hkv, D)
        k, v = torch.randn(shape, generator=g) + k_mean, torch.randn(shape, generator=g)
        if kv_dt == "fp8":
            k, v = (k / self.k_scale).clamp(-448, 448), (v / self.v_scale).clamp(-448, 448)
        k, v = k.to(TYPES[kv_dt]), v.to(TYPES[kv_dt])
        hide = torch.ones(self.num_pages, PAGE, dtype=torch.bool)
        at = 0
        for b, x in enumerate(kv):
            mine = ids[at:at + pages(x)]
            at += pages(x)
            table[b, :pages(x)] = mine.to(torch.int32)
            rows = torch.arange(pages(x) * PAGE).view(-1, PAGE) >= x
            hide[mine] = rows
        for t in (k, v):
            raw = t.view(torch.uint8) if kv_dt == "fp8" else t
            raw[hide] = 0x7f if kv_dt == "fp8" else math.nan
        self.q = torch.randn((self.T, Hq, D), generator=g).to(TYPES[q_dt]).to(device)
        self.k, self.v, self.table = k.to(device), v.to(device), table.to(device)
        cu = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
        self.cu = torch.from_numpy(cu).to(device)
        self.kv_len = torch.tensor(kv, dtype=torch.int32, device=device)
        self.out = torch.full(self.q.shape, 7.0, dtype=self.q.dtype, device=device)
        self.lse = torch.full((self.T, Hq), 7.0, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.q_dt, self.kv_dt = q_dt, kv_dt

    def workspace(self, q):
        n = q.qsa_chunk_attn_workspace_size(self.T, self.B, self.Hq, self.Hkv, self.D, self.k.dtype)
        return torch.full((n,), 0xff, dtype=torch.uint8, device=self.q.device)   # NaN all over

    def run(self, q, workspace=None, **kw):
        ws = self.workspace(q) if workspace is None else workspace
        return q.qsa_chunk_attn(self.q, self.k, self.v, self.table, self.cu, self.kv_len, self.out, workspace=ws,
                                k_scale=self.k_scale, v_scale=self.v_scale, lse=self.lse, dev_status=self.status, **kw)

    def keys(self, b, n, h):
        """Keys and values 0 .. n - 1 of request b and KV head h, in 64 bits."""
        idx = self.table[b, :pages(n)].long()
        k = self.k[idx, :, h].double().reshape(-1, self.D)[:n] * self.k_scale
        v = self.v[idx, :, h].double().reshape(-1, self.D)[:n] * self.v_scale
        return k, v

    def reference(self, sm_scale=None, skip=()):
        """(out, lse, tolerance of out, tolerance of lse).  skip: logical pages
        (b, page) whose tokens are left out.

        Tolerance of a logit: products of D terms summed in FP32 (D + 8
        roundings of 2^-24 of the sum of the terms' magnitudes; the scale, its
        product with the logit and the subtraction of the maximum are within
        the 8), plus the exponential's own 2^-22.  A probability is then off by
        that much relatively, plus one rounding to the type it meets V in
        (bf16 2^-8, fp16 2^-11, none in FP32), and both sums over n keys add
        (n + 16) 2^-24.  All act on A = sum_j p_j |v_j|; the output's own
        rounding comes on top."""
        G, D = self.Hq // self.Hkv, self.D
        scale = sm_scale if sm_scale else 1.0 / math.sqrt(D)
        dev = self.q.device
        out = torch.full(self.q.shape, 7.0, dtype=torch.float64, device=dev)
        lse = torch.full((self.T, self.Hq), 7.0, dtype=torch.float64, device=dev)
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        u_out = torch.finfo(self.q.dtype).eps / 2
        tc = self.q_dt == "bf16" and self.kv_dt != "f32"
        u_p = 0.0 if not tc else 2.0 ** -8 if self.kv_dt == "bf16" else 2.0 ** -11
        t0 = 0
        for b, (c, n) in enumerate(self.lens):
            L = max(int(self.kv_len[b]), 0)
            p = L - n + torch.arange(n, device=dev)
            rows = slice(t0, t0 + n)
            t0 += n
            if n == 0:
                continue
            if L == 0:
                out[rows], lse[rows] = 0, -math.inf
                continue
            hidden = torch.arange(L, device=dev)[None, :] > p[:, None]
            for pg in [x for y, x in skip if y == b]:
                hidden[:, pg * PAGE:(pg + 1) * PAGE] = True
            for h in range(self.Hkv):
                heads = slice(h * G, h * G + G)
                k, v = self.keys(b, L, h)
                x = self.q[rows, heads].double()
                s = torch.einsum("ngd,ld->ngl", x, k) * scale
                mag = torch.einsum("ngd,ld->ngl", x.abs(), k.abs()) * abs(scale)
                s = s.masked_fill(hidden[:, None], -math.inf)
                mag = mag.masked_fill(hidden[:, None], 0).amax(-1)
                z = torch.logsumexp(s, -1)
                pr = torch.exp(s - z[..., None])
                pr = torch.where(torch.isneginf(z)[..., None], 0.0, pr)
                # a token a row does not see adds nothing, whatever it holds
                w = torch.where(hidden[:, None, :, None], 0.0, pr[..., None] * v) if not torch.isfinite(v).all() else None
                o = w.sum(2) if w is not None else torch.einsum("ngl,ld->ngd", pr, v)
                A = w.abs().sum(2) if w is not None else torch.einsum("ngl,ld->ngd", pr, v.abs())
                logit = (D + 8) * 2.0 ** -24 * mag + 2.0 ** -22
                sums = (L + 16) * 2.0 ** -24
                rel = u_p + 2 * logit + 2 * sums
                out[rows, heads], lse[rows, heads] = o, z
                tol[rows, heads] = rel[..., None] * A + u_out * (o.abs() + rel[..., None] * A) + 1e-30
                ltol[rows, heads] = logit + sums + 2.0 ** -22 * (z.abs() + 1)
        return out, lse, tol, ltol

    def check(self, ref=None, status=0, **kw):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        out, lse, tol, ltol = self.reference(**kw) if ref is None else ref
        got, glse = self.out.double(), self.lse.double()
        for name, x, y, t in (("out", got, out, tol), ("lse", glse, lse, ltol)):
            odd = ~torch.isfinite(y)
            assert torch.equal(torch.isnan(x), torch.isnan(y)), f"{name}: NaN at other places"
            same = odd & ~torch.isnan(y)
            assert torch.equal(x[same], y[same]), f"{name}: infinities at other places"
            over = ((x - y).abs() - t)[~odd]
            assert over.numel() == 0 or float(over.max()) <= 0, \
                f"{name}: off by {float((x - y).abs()[~odd].max()):.3e}, past the tolerance by {float(over.max()):.3e}"
