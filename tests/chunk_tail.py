"""What FP16 probabilities below the type's normal range add to the tolerance of
the chunk attention over an FP8 cache."""
import torch

from chunk_utils import pages


def with_fp16_tail(b, ref):
    """`ref` (a Batch's reference) with the tolerance of `out` widened by the
    absolute rounding of small probabilities.

    Over an FP8 cache a probability meets V in FP16, as P = 2^(x - m).  The
    reference m moves to 7 below the largest logit (base 2) whenever that has
    outgrown it, so the largest P of every part of a row is 2^7 or more.  A P
    below 2^-14 is subnormal: it is rounded by up to half of 2^-24 whatever its
    own size, and one below 2^-25 becomes 0.  Both are at most 2^-25, 2^-32 of
    the part's largest P and so of the row's largest probability, which is at
    most 1: over the tokens a row sees this adds 2^-32 sum_j |v_j| (1.001 for the
    roundings of x and m themselves), and the output's rounding on top."""
    out, lse, tol, ltol = ref
    if b.kv_dt != "fp8" or b.q_dt != "bf16":
        return ref
    G, u = b.Hq // b.Hkv, 1 + torch.finfo(b.q.dtype).eps / 2
    tol, t0 = tol.clone(), 0
    for r, (_, n) in enumerate(b.lens):
        L = max(int(b.kv_len[r]), 0)
        if n and L:
            ids = b.table[r, :pages(L)].long()
            v = (b.v[ids].double() * b.v_scale).abs().nan_to_num(0, 0, 0).reshape(-1, b.Hkv, b.D)[:L].cumsum(0)
            p = (L - n + torch.arange(n, device=v.device))
            seen = torch.where((p >= 0)[:, None, None], v[p.clamp(min=0)], 0.0)
            tol[t0:t0 + n] += 1.001 * 2.0 ** -32 * u * seen.repeat_interleave(G, dim=1)
        t0 += n
    return out, lse, tol, ltol
