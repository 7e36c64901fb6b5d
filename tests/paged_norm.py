"""How far an attention output may be from the 64-bit one, row by row.

Every operand rounding of the kernels is at most half a step of fp16, u = 2^-11,
and different for every token and channel, so the errors of one output row add
up like independent ones.  With normalised weights w, values v, zero points z,
output o = sum_t w_t v_t, the variance of channel c's error is at most

    sum_t w_t^2 [ S_t (v_tc - o_c)^2 + u^2 m_tc^2 + u^2 v_tc^2 + a^2 ]

  S_t   variance of the score: scale^2 sum_c q_c^2 (u^2 k_tc^2 + a^2) for the key
        operand, u^2 scale^2 sum_c (q_c k_tc)^2 for the query's, and the fp32 sums,
        (2^-21 |scale| sum_c |q_c k_tc|)^2
  m_tc  what the weight operand multiplies: v, or v - z where the zero points are
        summed apart; the larger
  v_tc  the value operand
  a     half of fp16's smallest step, 2^-25: what rounding a subnormal may cost

A row's error, its norm over the channels, passes KAPPA = 6 deviations with a
probability of e^-18 or so (bounded errors, sub-Gaussian).  To this come the
output's own rounding (half a step of its type, element by element, never below
half its smallest) and fp16's
absolute step at the weights: one held below 2^-14 is off by up to 2^-25 instead
of u relative.
  Chunks hold the row's largest weight at 2^4 or more, so a weight below 2^-18 of
  it adds at most 2^-29 of it times the group's largest m.
  Few rows hold weight times value scale at 2^11 or more where both are the
  largest, so a product below 2^-25 of that adds at most 2^-36 of the largest
  weight times all groups' largest m.
A row of zeros, or one 5 % too large, is outside wherever more than a few tokens
share the weight.
"""
import numpy as np
import torch

from paged_util import GROUP, quantize, values

U = 2.0 ** -11
KAPPA = 6.0
A = 2.0 ** -25


def held(case, which, b, device):
    """(values, zero points, scales) of sequence b's tokens in 64 bits [t][h][d]."""
    codes, s, z = quantize(case.K[b] if which == "k" else case.V[b], case.bits)
    wide = lambda y: torch.from_numpy(np.repeat(y.astype(np.float64), GROUP, -1)).to(device)  # noqa: E731
    return torch.from_numpy(values(codes, s, z)).to(device).double(), wide(z), wide(s)


def check_rows(case, out, scale=None, gone=None, by_group=False, only=None, chunks=True):
    """Asserts that every real row of `out` is within the bound; returns the
    largest fraction of it that was used.  gone[b]: positions of sequence b that
    are not there (a page that does not exist).  by_group: the norm and the bound
    of each group of 32 channels by itself.  only: these sequences.
    chunks: whether some rows may be the chunk kernel's."""
    rg, d, dev = case.hq // case.hkv, case.d, out.device
    part = GROUP if by_group else d
    norm = lambda x: x.unflatten(-1, (-1, part)).norm(dim=-1)  # noqa: E731
    scale = d ** -0.5 if scale is None else scale
    half_step = torch.finfo(case.dtype).eps / 2
    tiny = half_step * torch.finfo(case.dtype).tiny + 1e-12
    assert torch.isfinite(out[:int(case.cu[-1])].float()).all()
    worst = 0.0
    for b, n in enumerate(case.new):
        if n == 0 or (only is not None and b not in only):
            continue
        at, kv = int(case.cu[b]), max(case.kv[b], 0)
        got = out[at:at + n].double().unflatten(1, (case.hkv, rg)).transpose(0, 1)  # [H][n][rg][d]
        if kv == 0:
            assert (got == 0).all()
            continue
        q = torch.from_numpy(case.q[at:at + n]).to(dev).double()
        q = q.unflatten(1, (case.hkv, rg)).transpose(0, 1)
        K, _, _ = held(case, "k", b, dev)
        V, Z, C = held(case, "v", b, dev)
        t = torch.arange(kv, device=dev)
        hidden = t[None] > (case.kv[b] - n + torch.arange(n, device=dev))[:, None]
        if gone and gone.get(b):
            hidden[:, list(gone[b])] = True
        hidden = hidden[:, None]
        for h in range(case.hkv):
            k, v = K[:, h], V[:, h]
            m2 = torch.maximum(v * v, (v - Z[:, h]) ** 2)
            s = (scale * (q[h] @ k.T)).masked_fill(hidden, -np.inf)             # [n][rg][t]
            w = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300))
            total = w.sum(-1, keepdim=True)
            w = w / torch.where(total > 0, total, 1.0)
            o = w @ v
            S = scale ** 2 * ((q[h] ** 2) @ (2 * U * U * k ** 2 + A * A).T
                              + (2.0 ** -21 * (q[h].abs() @ k.abs().T)) ** 2)
            a = w * w * S
            var = (a @ (v * v) - 2 * o * (a @ v) + o * o * a.sum(-1, keepdim=True)).clamp(min=0)
            var = var + U * U * ((w * w) @ (m2 + v * v + (A / U) ** 2))
            # the weights that may be below fp16's normal range, group by group
            top = w.amax(-1, keepdim=True)
            absolute = []
            for c in range(0, d, GROUP):
                size = C[:, h, c] / C[:, h].amax().clamp(min=1e-30)
                few_small = ((w * size < 2.0 ** -25 * top) & ~hidden).sum(-1)
                small = ((w < 2.0 ** -18 * top) & ~hidden).sum(-1) if chunks else 0
                each = (2.0 ** -36 * few_small * m2.amax().sqrt()
                        + 2.0 ** -29 * small * m2[:, c:c + GROUP].amax().sqrt())
                absolute.append(each * top[..., 0] * GROUP ** 0.5)
            absolute = torch.stack(absolute, -1).unflatten(-1, (d // part, -1)).norm(dim=-1)
            bound = (KAPPA * var.unflatten(-1, (-1, part)).sum(-1).sqrt() + half_step * norm(o)
                     + tiny * part ** 0.5 + absolute)
            use = float((norm(got[h] - o) / bound).max())
            assert use <= 1.0, "sequence %d head %d: %.2f of the bound" % (b, h, use)
            worst = max(worst, use)
    return worst
