"""Router inputs whose order 32-bit scores get wrong unseen where each gap is held against its two neighbours' errors alone:
choices of small scores without a bias, whose 32-bit values are nearly exact, beside large scores that a bias cancels, whose
32-bit values are off by 2^-25 and more."""
import numpy as np


def logit(p):
    return np.log(p / (1.0 - p))


def cancelled_scores(M, E, topk, score, seed):
    """logits [M][E] and bias [E] (fp32): topk + 1 small scores per row, a few times further apart than their own 32-bit errors,
    and one of E / 4 large scores with a bias that brings it near the last place; the rest far below.  (Softmax: the last
    expert takes what the others leave of the sum of 1, and its bias keeps it out of the choice.)"""
    rng = np.random.default_rng(seed)
    gap, near = (1e-8, 2e-8) if score == "sigmoid" else (1.5e-7, 1e-7)
    p = np.full((M, E), 1e-9)
    bias = np.zeros(E, np.float32)
    bias[E - 1] = -1.0
    large = rng.permutation(E - 1)[:E // 4]
    small = np.setdiff1d(np.arange(E - 1), large)
    bias[large] = -rng.uniform(0.5, 0.9, len(large))
    for m in range(M):
        steps = 1e-3 * (1 + rng.random()) - np.cumsum(rng.uniform(gap / 4, gap, topk + 1))
        p[m, rng.permutation(small)[:topk + 1]] = steps
        e = rng.choice(large)
        p[m, e] = steps[topk - 1] + rng.uniform(-near, near) - np.float64(bias[e])
        p[m, E - 1] = 1.0 - p[m, :E - 1].sum()
    return (logit(p) if score == "sigmoid" else np.log(p)).astype(np.float32), bias


def cancelled_groups(M, groups, per, seed):
    """logits [M][groups * per] and bias: in a quarter of the groups two biases of about +-1000 cancel, so that their sum is off
    by 2^-14 in 32 bits; every group's sum is 1.2 but for 10^-5 times a few units."""
    rng = np.random.default_rng(seed)
    E = groups * per
    p = rng.uniform(0.05, 0.2, (M, groups, per))
    bias = np.zeros((groups, per), np.float32)
    wide = rng.permutation(groups)[:max(1, groups // 4)]
    total = 1.2 + 1e-5 * rng.uniform(-4, 4, (M, groups))
    first = rng.uniform(0.5, 0.7, (M, groups))
    for g in range(groups):
        a, b = rng.permutation(per)[:2]
        p[:, g, a] = first[:, g]
        p[:, g, b] = total[:, g] - first[:, g]
        if g in wide:
            bias[g] = -2000.0
            bias[g, a] = 1000.0 + rng.integers(-3, 4)
            bias[g, b] = -bias[g, a]
    return logit(p).reshape(M, E).astype(np.float32), bias.reshape(E)
