"""How far an attention output may be from the 64-bit one, row by row.

Every operand rounding of the kernels is at most half a step of fp16, u = 2^-11,
and different for every token and channel, so the errors of one output row add
up like independent ones.  With normalised weights w, values v, zero points z,
output o = sum_t w_t v_t, the variance of channel c's error is at most

    sum_t w_t^2 [ S_t (v_tc - o_c)^2 + u^2 m_tc^2 + u^2 v_tc^2 ]

  S_t   variance of the score: u^2 scale^2 sum_c (q_c k_tc)^2 for the key operand,
        as much again for the query's, and the fp32 sums, (2^-21 |scale| sum_c
        |q_c k_tc|)^2
  m_tc  what the weight operand multiplies: v, or v - z where the zero points are
        summed apart; the larger
  v_tc  the value operand

A row's error, its norm over the channels, passes KAPPA = 6 deviations with a
probability of e^-18 or so (bounded errors, sub-Gaussian).  To this come the
output's own rounding (half a step of its type, element by element) and, for
weights below 2^-14 of the row's largest, FLOOR of the largest weight times the
largest m: fp16's absolute step, below the range that the kernels leave above it.
A row of zeros, or one 5 % too large, is outside wherever more than a few tokens
share the weight.
"""
import numpy as np
import torch

from paged_util import GROUP, quantize, values

U = 2.0 ** -11
KAPPA = 6.0
FLOOR = 2.0 ** -25


def held(case, which, b, device):
    """(values, zero points) of sequence b's tokens in 64 bits [t][h][d]."""
    codes, s, z = quantize(case.K[b] if which == "k" else case.V[b], case.bits)
    x = torch.from_numpy(values(codes, s, z)).to(device).double()
    return x, torch.from_numpy(np.repeat(z.astype(np.float64), GROUP, -1)).to(device)


def check_rows(case, out, scale=None, gone=None, floor=FLOOR):
    """Asserts that every real row of `out` is within the bound; returns the
    largest fraction of it that was used.  gone[b]: positions of sequence b that
    are not there (a page that does not exist)."""
    rg, d, dev = case.hq // case.hkv, case.d, out.device
    scale = d ** -0.5 if scale is None else scale
    half_step = torch.finfo(case.dtype).eps / 2
    assert torch.isfinite(out[:int(case.cu[-1])].float()).all()
    worst = 0.0
    for b, n in enumerate(case.new):
        if n == 0:
            continue
        at, kv = int(case.cu[b]), max(case.kv[b], 0)
        got = out[at:at + n].double().unflatten(1, (case.hkv, rg)).transpose(0, 1)  # [H][n][rg][d]
        q = torch.from_numpy(case.q[at:at + n]).to(dev).double()
        q = q.unflatten(1, (case.hkv, rg)).transpose(0, 1)
        K, _ = held(case, "k", b, dev)
        V, Z = held(case, "v", b, dev)
        t = torch.arange(kv, device=dev)
        hidden = t[None] > (case.kv[b] - n + torch.arange(n, device=dev))[:, None]
        if gone and gone.get(b):
            hidden[:, list(gone[b])] = True
        for h in range(case.hkv):
            k, v = K[:, h], V[:, h]
            m2 = torch.maximum(v * v, (v - Z[:, h]) ** 2)
            s = scale * (q[h] @ k.T)                                            # [n][rg][t]
            w = torch.exp((s - s.masked_fill(hidden[:, None], -np.inf)
                           .amax(-1, keepdim=True).clamp(min=-1e300)).masked_fill(
                               hidden[:, None], -np.inf)) if kv else s
            total = w.sum(-1, keepdim=True)
            w = w / torch.where(total > 0, total, 1.0)
            o = w @ v
            S = scale ** 2 * (2 * U * U * ((q[h] ** 2) @ (k ** 2).T)
                              + (2.0 ** -21 * (q[h].abs() @ k.abs().T)) ** 2)
            w2 = w * w
            a = w2 * S
            var = (a @ (v * v) - 2 * o * (a @ v) + o * o * a.sum(-1, keepdim=True)).clamp(min=0)
            var = var + U * U * (w2 @ (m2 + v * v))
            top = w.amax(-1, keepdim=True) if kv else torch.zeros_like(total)
            small = ((w < 2.0 ** -14 * top) & ~hidden[:, None]).sum(-1)
            big = m2.amax().sqrt() if kv else 0.0
            bound = (KAPPA * var.sum(-1).sqrt() + half_step * o.norm(dim=-1)
                     + floor * small * top[..., 0] * big * d ** 0.5 + 1e-7)
            err = (got[h] - o).norm(dim=-1)
            use = float((err / bound).max())
            assert use <= 1.0, "sequence %d head %d: %.2f of the bound" % (b, h, use)
            worst = max(worst, use)
    return worst
