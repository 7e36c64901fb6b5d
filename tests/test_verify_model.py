"""The tests' own form of draft verification: worked examples, and the property that
the method is for: whatever the drafts, tokens are distributed as the target's."""
import numpy as np

from verify_util import softmax, verify


def one(logits, tokens, draft, T, u, e):
    x = np.array(logits, float)
    n = len(x)
    d = None if draft is None else np.array(draft, float)
    return verify(x, np.array(tokens), np.array([0, n]), d, None if T is None else np.array([T]),
                  np.array(u, float), np.array([e], float))[0]


def test_worked_example():
    # p = (1/2, 1/4, 1/4), q = (1/4, 1/2, 1/4); draft 1 stays while u / 2 < 1/4
    p, q = np.log([2, 1, 1]), np.log([1, 2, 1])
    em, lp, close = one([p, p], [9, 1], [q, q], 1.0, [0.4, 0], [1, 1, 1])
    assert em == [1, 0] and not close
    assert np.allclose(lp, np.log([0.25, 0.5]))
    # refused: what is left is (1/4, 0, 0)
    em, _, _ = one([p, p], [9, 1], [q, q], 1.0, [0.6, 0], [100, 1, 1])
    assert em == [0]
    # certain drafts: u < 1/4; what is left is (1/2, 0, 1/4)
    assert one([p, p], [9, 1], None, 1.0, [0.2, 0], [1, 1, 1])[0] == [1, 0]
    assert one([p, p], [9, 1], None, 1.0, [0.3, 0], [3, 1, 1])[0] == [2]
    # greedy, ties to the lowest index
    assert one([[1, 1, 0], [0, 2, 2]], [9, 0], None, None, [0, 0], [1] * 3)[0] == [0, 1]
    assert one([[1, 1, 0], [0, 2, 2]], [9, 1], None, None, [0, 0], [1] * 3)[0] == [0]
    # nothing left at all
    assert one([[-np.inf] * 3], [9], None, 1.0, [0], [1] * 3)[0] == [-1]


def test_tokens_are_the_targets():
    rng = np.random.default_rng(0)
    V, N, T = 6, 40000, 0.8
    x, y = rng.standard_normal(V), rng.standard_normal(V)
    p, q = softmax(x, T)[0], softmax(y, T)[0]
    drafts = rng.choice(V, N, p=q)
    u, e = rng.random((N, 2)), rng.exponential(size=(N, V))
    first = np.zeros(V)
    for i in range(N):
        em, _, _ = one([x, x], [0, drafts[i]], [y, y], T, u[i], e[i])
        first[em[0]] += 1
    # a count's deviation is sqrt(N p (1 - p)) < 100; six of them
    assert (np.abs(first - N * p) < 600).all()
