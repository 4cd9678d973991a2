"""Plain 64-bit restatements of the latent cache's attention and derived error
bounds, for the GPU tests."""
import math

import torch

# half a step of each type, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def attend(q, k, v, limit, scale):
    """q [T, H, D], k [n, H or 1, D], v [n, H or 1, Dv] in float64; row t sees the
    first limit[t] keys.  Returns out, lse, sum_j w_j |v_j| (the weight that a
    relative error of every w_j puts on out) and the largest logit error unit
    scale * sum_d |q_d k_d|."""
    n = k.shape[0]
    t, h = q.shape[:2]
    if n == 0 or t == 0:
        z = torch.zeros(t, h, v.shape[2], dtype=torch.float64)
        return z, torch.full((t, h), -math.inf, dtype=torch.float64), z, torch.zeros(t, h, dtype=torch.float64)
    k, v = k.expand(n, h, k.shape[2]), v.expand(n, h, v.shape[2])
    s = scale * torch.einsum("thd,nhd->thn", q, k)
    size = scale * torch.einsum("thd,nhd->thn", q.abs(), k.abs())
    hidden = torch.arange(n)[None] >= limit[:, None]
    s = s.masked_fill(hidden[:, None], -math.inf)
    size = size.masked_fill(hidden[:, None], 0.0)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = e.sum(-1, keepdim=True)
    w = e / torch.where(l > 0, l, 1.0)
    v = torch.where((limit.max() > torch.arange(n))[:, None, None], v, 0.0)
    return (torch.einsum("thn,nhd->thd", w, v), (torch.log(l) + m).squeeze(-1),
            torch.einsum("thn,nhd->thd", w, v.abs()), size.amax(-1))


def bounds(ref, lse, absolute, size, n, d, dtype):
    """How far a kernel may be from `ref` and `lse` when logits are summed in
    fp32 (d terms, so at most d roundings of 2^-24 of the running magnitude,
    doubled for tensor-core sums that truncate), weights are rounded once to the
    cache's type, sums over n keys run in fp32 and the result is rounded once.
    A logit error of x changes every weight by a factor within e^x, and the sum
    too: 2x on out, x on lse."""
    logit = 2.0 * d * 2.0 ** -24 * size + 2.0 ** -21  # and the exponential's own error
    logit = logit + 2.0 ** -23 * lse.abs().nan_to_num(0.0, 0.0, 0.0)
    acc = 2.0 * (n + 8) * 2.0 ** -24
    half = HALF_STEP[dtype]
    rel = 2.0 * logit[..., None] + acc + half
    small = n * 2.0 ** -25 if dtype == torch.float16 else 0.0  # weights below fp16's least step
    out = rel * absolute + half * (ref.abs() + rel * absolute) + small * absolute.amax(-1, keepdim=True)
    if dtype == torch.float16:
        out = out + 2.0 ** -25  # the result may itself be below the least step
    return out, logit + acc
