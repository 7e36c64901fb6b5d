"""Draft verification in 64 bits for the tests, sequence by sequence (include/kvq.h,
kvq_verify_drafts).

Every decision is a comparison of positive numbers; the kernel computes each side in
fp32 to within a few 2^-24.  MARGIN = 2e-5 (relative) is what a decision has to have
to be the same there: p and q each are off by at most 2^-22 (the exponential), 2 *
2^-24 (its argument's rounding near the maximum, where the weight is) and the sum's
share of about 40 roundings, 2^-19 together; the test and the race multiply and
divide a few such numbers, and p - q magnifies the error of p by p / (p - q).
A sequence with a closer one is `close` from there on, and may be either.
"""
import numpy as np
import torch

MARGIN = 2e-5
FLOOR = 2.0 ** -126


def softmax(x, T):
    """Probabilities and their logarithms, masked logits at 0; None: nothing left."""
    x = np.where(np.isnan(x), -np.inf, x)
    x = np.minimum(x, 3e38)
    if not (x > -np.inf).any():
        return None
    t = (x - x.max()) / T
    e = np.exp(t)
    with np.errstate(divide="ignore"):
        return e / e.sum(), t - np.log(e.sum())


def first_largest(score, error):
    """(index, whether another may be as large): 64-bit scores and their error."""
    i = int(np.argmax(score))
    rival = score + error
    rival[i] = -1
    return i, bool((rival >= score[i] - error[i]).any()) if score[i] > 0 else True


def race(w, e, error):
    """The drawn index of weights w; error: absolute, of each."""
    ok = ~np.isnan(e)
    inv = np.where(ok, 1.0 / np.maximum(np.where(ok, e, 1.0), FLOOR), 0.0)
    if not (w * inv > 0).any():
        return -1, False
    return first_largest(w * inv, error * inv)


def verify(logits, tokens, cu, draft, temperature, uniform, noise):
    """numpy arrays (logits fp64) -> per sequence (tokens, logprobs, close): emitted
    tokens, their log probabilities, and whether a decision was too near to call
    (then the tokens up to there are right)."""
    V = logits.shape[1]
    out = []
    for b in range(len(cu) - 1):
        n, r = int(cu[b + 1] - cu[b]), int(cu[b])
        T = 0.0 if temperature is None else float(temperature[b])
        greedy = not T > 0
        em, lp, close = [], [], False
        for i in range(n):
            got = softmax(logits[r + i], 1.0 if greedy else T)
            p, logp = got if got else (np.zeros(V), np.full(V, -np.inf))
            c = int(tokens[r + i + 1]) if i < n - 1 else -1
            stay = False
            if greedy:
                t = int(np.argmax(p)) if got else -1
                stay = i < n - 1 and t == c and got is not None
            else:
                q = np.zeros(V)
                if i < n - 1 and 0 <= c < V:
                    if draft is not None:
                        have = softmax(draft[r + i], T)
                        q = have[0] if have else q
                    else:
                        q[c] = 1.0
                    with np.errstate(divide="ignore"):
                        lq = np.log(q[c]) if draft is None or not have else have[1][c]
                        left = np.log(np.float64(uniform[r + i])) + lq
                    stay = bool(left < logp[c])
                    with np.errstate(invalid="ignore"):
                        close |= bool(abs(left - logp[c]) < MARGIN) and got is not None
                if stay:
                    t = c
                else:
                    e = noise[b].astype(np.float64)
                    rest = np.maximum(p - q, 0) if i < n - 1 else p
                    error = MARGIN * (p + q)
                    if i < n - 1 and draft is None and 0 <= c < V:
                        rest, error = p.copy(), MARGIN * p
                        rest[c] = error[c] = 0.0
                    t, near = race(rest, e, error)
                    if t < 0 or not (rest > error).any():
                        near |= bool((error > 0).any()) and bool((rest > 0).any())
                        t2, n2 = race(p, e, MARGIN * p)
                        t = t2 if t < 0 else t
                        near |= n2
                    close |= near and got is not None
            em.append(t)
            lp.append(logp[t] if t >= 0 else 0.0)
            if close or not stay:
                break
        out.append((em, lp, close))
    return out


def log_bound(lp):
    """ln p = (x - m) / T - ln s: s to about 100 roundings (2^-24) relative, 2 ulp of
    the logarithm of s (up to ln V), the result's rounding."""
    return 100 * 2.0 ** -24 + 2 * 2.0 ** -23 * 12 + abs(lp) * 2.0 ** -22


def check(got, want, cu, tokens, allow_close=0.25):
    """Outputs of the call against verify()'s; padding and close sequences apart."""
    out, accepted, dropped, logs = (x.cpu().numpy() for x in got)
    n_close = 0
    for b, (em, lp, close) in enumerate(want):
        n, r = int(cu[b + 1] - cu[b]), int(cu[b])
        mine = out[r:r + n]
        sure = em[:-1] if close else em
        n_close += close
        assert list(mine[:len(sure)]) == sure, "sequence %d" % b
        assert accepted[b] + dropped[b] == max(n - 1, 0)
        if n:
            k = int(accepted[b])
            assert (mine[:k] == tokens[r + 1:r + 1 + k]).all()
            assert (mine[k + 1:] == -1).all() and (logs[r:r + n][mine < 0] == 0).all()
            if not close:
                assert k == len(em) - 1
        for i, x in enumerate(lp[:len(sure)]):
            assert abs(logs[r + i] - x) <= log_bound(x), "sequence %d row %d: %g, %g" % (
                b, i, logs[r + i], x)
    assert n_close <= allow_close * len(want) + 1


def call(verifier, logits, tokens, cu, draft=None, temperature=None, uniform=None, noise=None,
         **kw):
    return verifier.verify(logits, tokens, cu, draft, temperature, uniform, noise, **kw)


def wide(t):
    return None if t is None else t.double().cpu().numpy()


def expected(logits, tokens, cu, draft=None, temperature=None, uniform=None, noise=None):
    return verify(wide(logits), tokens.cpu().numpy(), cu.cpu().numpy(), wide(draft),
                  wide(temperature), wide(uniform), wide(noise))
