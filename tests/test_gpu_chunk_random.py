"""Random batches of the chunk attention: head groups of 1 to 16, every kernel,
decode steps to prompts, up to 200 requests, here and there a value that is not
finite; against the plain form in 64 bits, and bit-equal from run to run."""
import math
import random

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


def random_batch(rng):
    G, Hkv = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 8, 11, 12, 12, 16, 16]), rng.choice([1, 1, 2, 2, 3, 4])
    D = rng.choice([64, 128, 256, 256])
    q_dt, kv_dt = rng.choice([("bf16", "bf16"), ("bf16", "fp8"), ("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32")])
    n_req = rng.choice([1, 1, 2, 3, 5, 9, 17, 40, 90, 200])
    mode = rng.choice(["decode", "drafts", "chunk", "mixed", "mixed", "prompt"])
    lens = []
    for _ in range(n_req):
        old = int(rng.random() ** 3 * max(1, 40000 // n_req)) if rng.random() < 0.9 else rng.choice([0, 63, 64, 65, 127, 128])
        if mode == "decode":
            new = 1
        elif mode == "drafts":
            new = rng.randrange(0, 5)
        elif mode == "mixed":
            new = 1 if rng.random() < 0.7 else rng.randrange(0, max(2, 600 // n_req))
        else:
            new = rng.randrange(1, max(2, 1500 // n_req))
            old = 0 if mode == "prompt" else old
        lens.append((old, new))
    lens[0] = (lens[0][0], max(1, lens[0][1]))
    b = Batch(lens, G * Hkv, Hkv, D, q_dt, kv_dt, seed=rng.randrange(1 << 30), pad=rng.choice([0, 0, 3]))
    if rng.random() < 0.3:
        b.q.mul_(6)
    # the reference holds a request's every probability times every value then
    if rng.random() < 0.4 and max(n * G * (c + n) * D for c, n in lens) < 1 << 29:
        for _ in range(rng.randrange(1, 6)):
            r = rng.randrange(n_req)
            kv = sum(lens[r])
            if kv:
                p = max(0, kv - 1 - int(rng.random() ** 2 * kv)) if rng.random() < 0.5 else kv - 1
                at = int(b.table[r, p // 64]), p % 64, rng.randrange(Hkv), rng.randrange(D)
                if kv_dt == "fp8":
                    b.v.view(torch.uint8)[at] = rng.choice([0x7f, 0xff])
                else:
                    b.v[at] = math.nan
    return b


def check(q, rng):
    b = random_batch(rng)
    ws, ref = b.workspace(q), with_fp16_tail(b, b.reference())
    b.run(q, workspace=ws)
    b.check(ref=ref)
    raw = torch.int32 if b.q_dt == "f32" else torch.int16
    first, flse = b.out.clone(), b.lse.clone()
    for _ in range(4):
        b.run(q, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(first.view(raw), b.out.view(raw)) and torch.equal(flse.view(torch.int32), b.lse.view(torch.int32))


@pytest.mark.parametrize("seed", range(60))
def test_random_batches(q, seed):
    check(q, random.Random(seed))
