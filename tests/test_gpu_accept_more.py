"""Acceptance of drafted tokens: calls that test_gpu_accept leaves out."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_accept import Case, check, run  # noqa: E402


@pytest.mark.parametrize("seqs,vocab", [(1, 40), (5, 70001), (300, 257), (40, 70001)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_batches_of_one_row(seqs, vocab, dtype):
    """No statistics and no tests: the walk's first step is the exchange of
    its cluster, here with clusters of every size and more than run at once."""
    c = Case("chain", [1] * seqs, [0] * seqs, vocab, dtype, False, 1.0, seqs + vocab)
    first = check(c)
    for _ in range(20):
        for a, b in zip(run(c), first):
            assert np.array_equal(a, b)


def nearly_the_target(n, delta, seed):
    """Logits, their softmax p and a drafter's g whose residual max(p - g, 0)
    has a mass of 2 delta: half of it over the first n / 2 entries, where g =
    (1 - delta) p, half over the others, where g = 0, so that a cut c g that is
    off by a share e of itself moves the border between the halves by about
    e / (4 delta).  Entry n / 4 has g > p."""
    r = np.random.default_rng(seed)
    k = n // 2
    x = (r.standard_normal(n) * 0.3).astype(np.float32)
    z = np.exp(x.astype(np.float64))
    x[k:] += np.float32(np.log(delta * z[:k].sum() / z[k:].sum()))
    z = x.astype(np.float64)
    p = np.exp(z - z.max())
    p /= p.sum()
    g = p.copy()
    g[:k] *= 1 - delta
    g[k:] = 0.0
    g[k // 2] = 0.0
    g[k // 2] = 1 - g.sum()
    return x, p, g.astype(np.float32)


@pytest.mark.parametrize("n,delta,seed", [(301, 1e-3, 0), (301, 1e-4, 1), (301, 1e-4, 2), (2000, 1e-4, 2), (2000, 1e-3, 2),
                                          (131072, 1e-4, 3)])
def test_draws_next_to_a_border_after_a_rejection(n, delta, seed):
    """A drafter close to the target: the borders of what a rejection leaves are
    off by at most 1e-10 over its mass (weights off by 2^-32 of themselves,
    their sum's share of it some 5e-11), and numbers that far from a border, on
    either side, draw the oracle's token."""
    x, p, g = nearly_the_target(n, delta, seed)
    res = np.maximum(p - g.astype(np.float64), 0.0)
    mass = res.sum()
    c = np.cumsum(res) / mass
    off = 1e-10 / mass
    v = []
    for i in range(n // 2 - 9, n // 2 + 10):
        for side in (-1.0, 1.0):
            w = np.float32(c[i] + side * 1.5 * off)
            if np.abs(c - np.float64(w)).min() > off:
                v.append(w)
    assert len(v) >= 10
    case = Case("chain", [2] * len(v), [0] * len(v), n, "f32", True, 1.0, 0)
    rows = case.base.reshape(2 * len(v), n)
    rows[:] = torch.from_numpy(x)
    case.logits = rows.numpy().astype(np.float64)
    case.probs = np.tile(g, (2 * len(v), 1))
    case.tokens[:] = n // 2 // 2  # g > p there
    assert p[n // 4] < 0.9999 * g[n // 4]
    case.u[:] = 0.99999
    case.v = np.asarray(v, np.float32)
    got = check(case, close=off * 0.99)
    assert (got[0] == 1).all()
