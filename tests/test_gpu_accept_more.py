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
