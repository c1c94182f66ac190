"""The operators of a dense chunk step over the paged KV cache, as they are measured.

Three operators, in the order a serving step runs them:

  plan   block tables and slot maps from the request lengths: every new token's
         request, position and physical cache slot, and the page table grown
         from a list of free pages
  rope   rotary positions with one to three axes on the step's queries and
         keys, and the write of keys and values into the cache at those slots
  attn   causal attention of each request's new tokens over all of its cached
         tokens: prompts and chunks of them, single tokens, draft tokens

``run`` computes them in plain torch operations, or, where ``own`` is true,
with the library's calls.
"""
import math
import random

import torch

own = False

PAGE = 64
FP8_MAX = 448.0
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
SIZES = {"f32": 4, "bf16": 2, "fp8": 1}


# ---- cases ----------------------------------------------------------------------
#
# Lengths of a batch follow from the case alone: "new" and "old" are the ranges
# of a request's new and cached tokens, drawn (over their logarithm) from a
# generator seeded by "mix".

def listed():
    return [
        # one decode step's tables for the batch of the decode benchmark
        dict(name="plan_decode_b8", op="plan", B=8, new_lo=1, new_hi=1, old_lo=262143, old_hi=262143, pad=0, width=4096,
             mix=1),
        # a mixed step of many requests (decodes and chunks), padded to a captured size
        dict(name="plan_mixed_b256", op="plan", B=256, new_lo=1, new_hi=300, old_lo=0, old_hi=20000, pad=37, width=512,
             mix=2),
        # many prompts admitted at once: the largest tables
        dict(name="plan_prompts_b1000", op="plan", B=1000, new_lo=16, new_hi=1024, old_lo=0, old_hi=200, pad=0,
             width=1024, mix=3),
        # a decode step: 8 tokens, FP8 cache, a quarter of the head rotated
        dict(name="rope_decode_fp8", op="rope", B=8, new_lo=1, new_hi=1, old_lo=1, old_hi=20000, pad=0, Hq=16, Hkv=2,
             D=256, rot=64, axes=1, split="chunked", pairs="halves", x="bf16", kv="fp8", mix=4),
        # a prompt with images: three axes, interleaved, ragged
        dict(name="rope_image_bf16", op="rope", B=3, new_lo=300, new_hi=900, old_lo=0, old_hi=500, pad=11, Hq=24, Hkv=2,
             D=256, rot=64, axes=3, split="interleaved", pairs="halves", x="bf16", kv="bf16", mix=5),
        # float32 with adjacent pairs, the whole head rotated
        dict(name="rope_f32_d64", op="rope", B=5, new_lo=1, new_hi=700, old_lo=0, old_hi=100, pad=0, Hq=4, Hkv=1, D=64,
             rot=64, axes=2, split="chunked", pairs="adjacent", x="f32", kv="f32", mix=6),
        # the prefill chunk of the benchmark, the whole head rotated
        dict(name="rope_prefill_8192", op="rope", B=1, new_lo=8192, new_hi=8192, old_lo=57344, old_hi=57344, pad=0,
             Hq=24, Hkv=2, D=256, rot=256, axes=3, split="chunked", pairs="halves", x="bf16", kv="bf16", mix=7),
        # the decode batch of the benchmark, attending densely: one token each, FP8 cache
        dict(name="attn_decode_b8_262k_fp8", op="attn", B=8, new_lo=1, new_hi=1, old_lo=262143, old_hi=262143, pad=0,
             Hq=16, Hkv=2, D=256, x="bf16", kv="fp8", mix=8),
        # a ragged decode batch with drafts behind each token: 1 to 4 tokens a request
        dict(name="attn_drafts_b33_bf16", op="attn", B=33, new_lo=1, new_hi=4, old_lo=1, old_hi=16384, pad=5, Hq=16,
             Hkv=2, D=256, x="bf16", kv="bf16", mix=9),
        # a mixed step: decodes and chunks of several prompts, FP8 cache, 12 query heads on one KV head
        dict(name="attn_mixed_b9_fp8", op="attn", B=9, new_lo=1, new_hi=1500, old_lo=0, old_hi=9000, pad=3, Hq=12,
             Hkv=1, D=128, x="bf16", kv="fp8", mix=10),
        # a tiny float32 model's prompts
        dict(name="attn_f32_d64", op="attn", B=4, new_lo=40, new_hi=260, old_lo=0, old_hi=700, pad=0, Hq=4, Hkv=1, D=64,
             x="f32", kv="f32", mix=11),
        # the prefill chunk of the benchmark, dense: 8,192 new tokens behind 57,344 cached ones
        dict(name="attn_prefill_8192_65536", op="attn", B=1, new_lo=8192, new_hi=8192, old_lo=57344, old_hi=57344,
             pad=0, Hq=24, Hkv=2, D=256, x="bf16", kv="bf16", mix=12),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm."""
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1))) - 1))))


HEADS = ((16, 2), (24, 2), (12, 1), (6, 1), (3, 1), (4, 1), (8, 8))


def draw(rng):
    op = rng.choice(("plan", "rope", "rope", "attn", "attn", "attn"))
    mix = rng.randrange(1000, 1 << 20)
    if op == "plan":
        B = _spread(rng, 1, 1200)
        hi = _spread(rng, 1, max(1, 200000 // B))
        old = _spread(rng, 0, 60000)
        return dict(op=op, B=B, new_lo=_spread(rng, 0, hi), new_hi=hi, old_lo=_spread(rng, 0, old), old_hi=old,
                    pad=rng.choice((0, rng.randrange(200))), width=-(-(old + hi) // PAGE) + rng.randrange(40), mix=mix)
    Hq, Hkv = rng.choice(HEADS)
    x = rng.choice(("bf16", "bf16", "bf16", "f32"))
    D = rng.choice((64, 128, 256))
    kv = rng.choice(("bf16", "fp8")) if x == "bf16" else "f32"
    if op == "rope":
        B = _spread(rng, 1, 64)
        hi = _spread(rng, 1, 7000 // B)
        rot = rng.choice((D, D // 2, D // 4))
        return dict(op=op, B=B, new_lo=_spread(rng, 1, hi), new_hi=hi, old_lo=0, old_hi=_spread(rng, 0, 40000 // B),
                    pad=rng.choice((0, rng.randrange(30))), Hq=Hq, Hkv=Hkv, D=D, rot=rot, axes=rng.choice((1, 2, 3)),
                    split=rng.choice(("chunked", "interleaved")), pairs=rng.choice(("halves", "adjacent")), x=x, kv=kv,
                    mix=mix)
    B = _spread(rng, 1, 40)
    kind = rng.choice(("decode", "drafts", "chunk"))
    hi = 1 if kind == "decode" else rng.randrange(2, 9) if kind == "drafts" else _spread(rng, 2, 4000 // B)
    old = _spread(rng, 0, (600000 if kind != "chunk" else 60000) // B)
    if x == "f32":
        hi, old = min(hi, 300), min(old, 2000)
    return dict(op=op, B=B, new_lo=1 if kind != "chunk" else _spread(rng, 1, hi), new_hi=hi, old_lo=_spread(rng, 0, old),
                old_hi=old, pad=rng.choice((0, rng.randrange(9))), Hq=Hq, Hkv=Hkv, D=D, x=x, kv=kv, mix=mix)


def lengths(case):
    """(cached, new) tokens of every request."""
    rng = random.Random(case["mix"])
    return [(_spread(rng, case["old_lo"], case["old_hi"]), _spread(rng, case["new_lo"], case["new_hi"]))
            for _ in range(case["B"])]


# ---- inputs ---------------------------------------------------------------------

class State:
    pass


def _pages(n):
    return -(-n // PAGE)


def _store(x, kind, scale):
    """Values in a cache's storage type (FP8: codes of value / scale)."""
    if kind == "fp8":
        return (x / scale).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return x.to(DTYPES[kind])


def _cache(shape, kind, scale, g):
    out = torch.empty(shape, dtype=DTYPES[kind], device="cuda")
    step = max(1, (1 << 26) // max(1, math.prod(shape[1:])))
    for i in range(0, shape[0], step):
        out[i:i + step] = _store(torch.randn(out[i:i + step].shape, generator=g, device="cuda"), kind, scale)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ints = dict(dtype=torch.int32, device="cuda")
    lens = lengths(case)
    s = State()
    s.case, s.lens = case, lens
    B = case["B"]
    old = torch.tensor([c for c, _ in lens], **ints)
    new = torch.tensor([n for _, n in lens], **ints)
    used = sum(n for _, n in lens)
    s.T = max(1, used + case["pad"])
    if case["op"] == "plan":
        s.old, s.new = old, new
        have = sum(_pages(c) for c, _ in lens)
        grow = sum(_pages(c + n) - _pages(c) for c, n in lens)
        s.num_pages = have + grow + 100
        ids = torch.randperm(s.num_pages, generator=g, device="cuda").to(torch.int32)
        s.width = max(case["width"], max(_pages(c + n) for c, n in lens), 1)
        s.table = torch.full((B, s.width), -1, **ints)
        cols = torch.arange(s.width, device="cuda")
        mine = cols < ((old + PAGE - 1) // PAGE)[:, None]
        s.table[mine] = ids[:have]
        s.free = ids[have:].contiguous()
        s.cu = torch.empty(B + 1, **ints)
        s.kv_len = torch.empty(B, **ints)
        s.req, s.pos, s.slot = (torch.empty(s.T, **ints) for _ in range(3))
        s.taken = torch.empty(1, **ints)
        s.status = torch.zeros(1, **ints)
        return s
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    width = max(max(_pages(c + n) for c, n in lens), 1)
    total = sum(_pages(c + n) for c, n in lens)
    s.num_pages = total + 3
    ids = torch.randperm(s.num_pages, generator=g, device="cuda").to(torch.int32)
    s.table = torch.full((B, width), -1, **ints)
    mine = torch.arange(width, device="cuda") < ((old + new + PAGE - 1) // PAGE)[:, None]
    s.table[mine] = ids[:total]
    s.k_scale, s.v_scale = (4.5 / FP8_MAX, 5.0 / FP8_MAX) if case["kv"] == "fp8" else (1.0, 1.0)
    s.k_pages = _cache((s.num_pages, PAGE, Hkv, D), case["kv"], s.k_scale, g)
    s.v_pages = _cache((s.num_pages, PAGE, Hkv, D), case["kv"], s.v_scale, g)
    s.status = torch.zeros(1, **ints)
    cu = [0]
    for _, n in lens:
        cu.append(cu[-1] + n)
    if case["op"] == "rope":
        # queries, keys and values lie in one projection's output, row by row
        qkv = torch.randn((s.T, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(DTYPES[case["x"]])
        s.q = qkv[:, :Hq * D].view(s.T, Hq, D)
        s.k = qkv[:, Hq * D:(Hq + Hkv) * D].view(s.T, Hkv, D)
        s.v = qkv[:, (Hq + Hkv) * D:].view(s.T, Hkv, D)
        req = torch.repeat_interleave(torch.arange(B, device="cuda"), new.long())
        first = torch.tensor(cu[:-1], device="cuda")
        p = (old.long()[req] + torch.arange(used, device="cuda") - first[req])
        slot = s.table[req, p // PAGE].long() * PAGE + p % PAGE
        s.slot = torch.full((s.T,), -1, **ints)
        s.slot[:used] = slot.to(torch.int32)
        s.pos = torch.zeros((case["axes"], s.T), **ints)
        s.pos[:, :used] = p.to(torch.int32)
        if case["axes"] > 1:   # images: the further axes run over rows and columns
            s.pos[1:, :used] += torch.randint(-40, 41, (case["axes"] - 1, used), generator=g, device="cuda",
                                              dtype=torch.int32)
            s.pos.clamp_(min=0)
        half = case["rot"] // 2
        s.inv_freq = (1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        s.sections = sections(case)
        s.q_out = torch.zeros((s.T, Hq, D), dtype=DTYPES[case["x"]], device="cuda")
        return s
    s.q = torch.randn((s.T, Hq, D), generator=g, device="cuda").to(DTYPES[case["x"]])
    s.cu = torch.tensor(cu, **ints)
    s.kv_len = (old + new).contiguous()
    s.out = torch.zeros((s.T, Hq, D), dtype=DTYPES[case["x"]], device="cuda")
    s.lse = torch.zeros((s.T, Hq), device="cuda")
    if own:
        from indexer_top_sparse_c4_b200 import qsa
        size = qsa.qsa_chunk_attn_workspace_size(s.T, B, Hq, Hkv, D, s.k_pages.dtype)
        s.workspace = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return s


def sections(case):
    """Frequencies of each axis (a third each, the first axis the rest)."""
    half = case["rot"] // 2
    if case["axes"] == 1:
        return (half, 0, 0)
    side = half // 3
    if case["axes"] == 2:
        return (half - side, side, 0)
    return (half - 2 * side, side, side)


# ---- one pass -------------------------------------------------------------------

def run(s):
    return {"plan": _plan, "rope": _rope, "attn": _attn}[s.case["op"]](s)


def _plan(s):
    if own:
        from indexer_top_sparse_c4_b200 import qsa
        qsa.qsa_chunk_plan(s.old, s.new, s.free, s.table, s.num_pages, s.cu, s.kv_len, s.req, s.pos, s.slot, s.taken,
                           dev_status=s.status)
        return [s.cu, s.kv_len, s.req, s.pos, s.slot, s.table, s.taken]
    B, T = s.case["B"], s.T
    old, new = s.old.long(), s.new.long()
    kv = old + new
    cu = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    cu[1:] = torch.cumsum(new, 0)
    has, need = (old + PAGE - 1) // PAGE, (kv + PAGE - 1) // PAGE
    grow = need - has
    base = torch.cumsum(grow, 0) - grow
    cols = torch.arange(s.width, device="cuda")
    fresh = (cols >= has[:, None]) & (cols < need[:, None])
    take = (base[:, None] + cols - has[:, None]).clamp(0, s.free.numel() - 1)
    s.table.copy_(torch.where(fresh, s.free[take], s.table))
    t = torch.arange(T, device="cuda")
    live = t < cu[B]
    req = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    pos = old[req] + t - cu[req]
    slot = s.table[req, (pos // PAGE).clamp(max=s.width - 1)].long() * PAGE + pos % PAGE
    req, pos, slot = (torch.where(live, v, -1).to(torch.int32) for v in (req, pos, slot))
    return [cu.to(torch.int32), kv.to(torch.int32), req, pos, slot, s.table, grow.sum().to(torch.int32).reshape(1)]


def _axis_of(case):
    """The axis each frequency takes its position from."""
    half, sec = case["rot"] // 2, sections(case)
    i = torch.arange(half, device="cuda")
    if case["split"] == "chunked":
        return (i >= sec[0]).long() + (i >= sec[0] + sec[1]).long()
    return torch.where((i % 3 == 1) & (i < 3 * sec[1]), 1, torch.where((i % 3 == 2) & (i < 3 * sec[2]), 2, 0))


def _rotated(x, cos, sin, case):
    """x [T, H, D] in 32 bits with its first rot values rotated."""
    x, rot, half = x.float(), case["rot"], case["rot"] // 2
    if case["pairs"] == "halves":
        a, b = x[..., :half], x[..., half:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], dim=-1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2), x[..., rot:]], dim=-1)


def _rope(s):
    c = s.case
    if own:
        from indexer_top_sparse_c4_b200 import qsa
        qsa.qsa_rope_write(s.q, s.k, s.v, s.pos, s.inv_freq, s.slot, s.q_out, s.k_pages, s.v_pages,
                           sections=s.sections, interleaved_axes=c["split"] == "interleaved",
                           adjacent_pairs=c["pairs"] == "adjacent", k_scale=s.k_scale, v_scale=s.v_scale,
                           dev_status=s.status)
        return [s.q_out, s.k_pages, s.v_pages]
    angle = s.pos[_axis_of(c)].double().T * s.inv_freq.double()
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    q_out = _rotated(s.q, cos, sin, c).to(s.q.dtype)
    k = _store(_rotated(s.k, cos, sin, c), c["kv"], s.k_scale)
    v = _store(s.v.float(), c["kv"], s.v_scale)
    # rows without a slot write the first row's values once more
    live = s.slot >= 0
    row = torch.where(live, torch.arange(s.T, device="cuda"), 0)
    at = s.slot[row].long()
    kind = torch.uint8 if c["kv"] == "fp8" else DTYPES[c["kv"]]
    s.k_pages.view(kind).view(-1, c["Hkv"], c["D"])[at] = k.view(kind)[row]
    s.v_pages.view(kind).view(-1, c["Hkv"], c["D"])[at] = v.view(kind)[row]
    return [torch.where(live[:, None, None], q_out, 0), s.k_pages, s.v_pages]


def _attn(s):
    c = s.case
    if own:
        from indexer_top_sparse_c4_b200 import qsa
        qsa.qsa_chunk_attn(s.q, s.k_pages, s.v_pages, s.table, s.cu, s.kv_len, s.out, workspace=s.workspace,
                           k_scale=s.k_scale, v_scale=s.v_scale, lse=s.lse, dev_status=s.status)
        return [s.out, s.lse]
    B, T, Hq, Hkv, D = c["B"], s.T, c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    N = max(n for _, n in s.lens)
    L = max(o + n for o, n in s.lens)
    cu, kv_len = s.cu.long(), s.kv_len.long()
    t = torch.arange(T, device="cuda")
    live = t < cu[B]
    req = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    # queries and cached tokens of the batch, padded to the longest request
    i = torch.arange(N, device="cuda")
    row = (cu[:-1, None] + i).clamp(max=T - 1)
    q = s.q[row].float().view(B, N, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * N, D)
    table = s.table.clamp(min=0).long()
    k = s.k_pages[table].flatten(1, 2)[:, :L].permute(0, 2, 3, 1).float()
    v = s.v_pages[table].flatten(1, 2)[:, :L].permute(0, 2, 1, 3).float()
    x = torch.matmul(q, k).mul_(s.k_scale / math.sqrt(D)).view(B, Hkv, G, N, L)
    pos = kv_len[:, None] - (cu[1:] - cu[:-1])[:, None] + i
    hidden = torch.arange(L, device="cuda") > pos[..., None]
    x.masked_fill_(hidden[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, G * N, L), v).view(B, Hkv, G, N, D) * (s.v_scale / total)
    lse = (top + total.log()).squeeze(-1)
    i = (t - cu[req]).clamp(max=N - 1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)[req, i]
    lse = lse.permute(0, 3, 1, 2).reshape(B, N, Hq)[req, i]
    return [torch.where(live[:, None, None], o, 0).to(s.out.dtype), torch.where(live[:, None], lse, 0)]


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    lens = lengths(case)
    used = sum(n for _, n in lens)
    if case["op"] == "plan":
        # lengths read; table entries read where new tokens share a page with
        # cached ones, pages taken and entered; three numbers a token
        grow = sum(_pages(c + n) - _pages(c) for c, n in lens)
        return {"bytes": 8 * case["B"] + 8 * (case["B"] + 1) + 8 * grow + 12 * (used + case["pad"]),
                "flops": 10 * used}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    x, kv = SIZES[case["x"]], SIZES[case["kv"]]
    if case["op"] == "rope":
        half = case["rot"] // 2
        return {"bytes": used * (2 * Hq * D * x + 2 * Hkv * D * (x + kv) + 4 * case["axes"] + 4) + 4 * half,
                "flops": used * half * (6 * (Hq + Hkv) + 20)}
    seen = sum(n * c + n * (n + 1) // 2 for c, n in lens)
    return {"bytes": used * Hq * (2 * D * x + 4) + 2 * sum(c + n for c, n in lens) * Hkv * D * kv,
            "flops": 4 * seen * Hq * D}


# ---- the definitions, in 64 bits ------------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn}[case["op"]](s)


def _exact_rope(s):
    """Each pair of a head as a complex number times exp(i * position * frequency)."""
    c = s.case
    half, rot = c["rot"] // 2, c["rot"]
    sec = s.sections
    names = []
    for i in range(half):
        if c["split"] == "chunked":
            names.append(0 if i < sec[0] else 1 if i < sec[0] + sec[1] else 2)
        else:
            names.append(1 if i % 3 == 1 and i < 3 * sec[1] else 2 if i % 3 == 2 and i < 3 * sec[2] else 0)
    pos = s.pos.double()
    phase = torch.stack([pos[a] * s.inv_freq[i].double() for i, a in enumerate(names)], dim=1)
    turn = torch.polar(torch.ones_like(phase), phase)[:, None]

    def turned(x):
        y = x.double().clone()
        even, odd = (slice(0, half), slice(half, rot)) if c["pairs"] == "halves" else (slice(0, rot, 2),
                                                                                       slice(1, rot, 2))
        z = torch.complex(y[..., even], y[..., odd]) * turn
        y[..., even], y[..., odd] = z.real, z.imag
        return y

    n = sum(m for _, m in s.lens)
    q = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    q[:n] = turned(s.q)[:n]
    if c["kv"] == "fp8":   # codes: a rounding of the value to 8 bits, which has no value in 64
        return [q, None, None]
    k, v = s.k_pages.double(), s.v_pages.double()
    at = s.slot[:n].long()
    k.view(-1, c["Hkv"], c["D"])[at] = turned(s.k)[:n]
    v.view(-1, c["Hkv"], c["D"])[at] = s.v[:n].double()
    return [q, k, v]


def _exact_attn(s):
    c = s.case
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    out = torch.zeros((s.T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s.T, Hq), dtype=torch.float64, device="cuda")
    t0 = 0
    for r, (o, n) in enumerate(s.lens):
        L = o + n
        ids = s.table[r, :_pages(L)].long()
        for h in range(Hkv):
            k = s.k_pages[ids, :, h].double().reshape(-1, D)[:L] * s.k_scale
            v = s.v_pages[ids, :, h].double().reshape(-1, D)[:L] * s.v_scale
            block = max(1, (1 << 28) // (G * max(L, 1)))
            for a in range(0, n, block):
                m = min(block, n - a)
                rows = slice(t0 + a, t0 + a + m)
                heads = slice(h * G, h * G + G)
                logits = torch.einsum("ngd,ld->ngl", s.q[rows, heads].double(), k) / math.sqrt(D)
                last = o + a + torch.arange(m, device="cuda")
                logits = logits.masked_fill(torch.arange(L, device="cuda")[None, None] > last[:, None, None], -math.inf)
                z = torch.logsumexp(logits, dim=-1)
                lse[rows, heads] = z
                out[rows, heads] = torch.einsum("ngl,ld->ngd", torch.exp(logits - z[..., None]), v)
        t0 += n
    return [out, lse]
