"""How far the inputs of the GPU acceptance tests keep from their borders: the
tests of children and the draw have errors of their own, so each has a
distance of its own.  Runs on the CPU, with the oracle in the kernel's place."""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle.step_oracle as so
import test_gpu_accept as gpu

# Tests of a child are fp32: statistics of up to 2^20 positive terms, each off by
# at most 2^-22, and the pieces' rescaling.  Without drafted probabilities the
# mass of the rejected siblings is such a sum too, and its error counts over
# what they left.  With them the later siblings meet fixed-point weights, off
# by 2^-32, over what the rejections left.
FP32, FIXED = 1e-5, 1e-9


def needed(case, before, left):
    return FIXED / left if case.probs is not None and before else FP32 / left


def decisions(case):
    for s in range(len(case.cu) - 1):
        a, b = int(case.cu[s]), int(case.cu[s + 1])
        if a == b:
            continue
        par = [int(x) for x in case.parent[a:b]] if case.kinds[s] else list(range(-1, b - a - 1))
        yield so.accept_decisions(case.logits[a:b], None if case.probs is None else case.probs[a:b], case.tokens[a:b],
                                  par, case.u[a:b], case.v[s], float(case.temperature[s]))


def margins(case):
    """The smallest test and draw of a case, each over what it has to keep."""
    tests, draws = [np.inf], [np.inf]
    for _, _, tried, (draw, left) in decisions(case):
        tests += [d / needed(case, *at) for d, *at in tried]
        draws.append(draw * left / FIXED)
    return min(tests), min(draws)


def combinations(fn):
    marks = [m for m in getattr(fn, "pytestmark", []) if m.name == "parametrize"]
    for values in itertools.product(*(m.args[1] for m in marks)):
        kw = {}
        for m, v in zip(marks, values):
            names = [n.strip() for n in m.args[0].split(",")]
            kw.update(zip(names, v if len(names) > 1 else [v]))
        yield kw


CHECKED = [gpu.test_chains, gpu.test_trees_with_odd_strides, gpu.test_batches_that_all_run_at_once_and_do_not,
           gpu.test_batches_whose_weights_fit_a_cluster_and_do_not, gpu.test_mixed_kinds_and_temperatures,
           gpu.test_many_siblings, gpu.test_a_chain_of_the_most_rows, gpu.test_ties_go_to_the_lowest_index,
           gpu.test_masked_vocabulary_and_peaked_rows]


@pytest.mark.parametrize("fn", CHECKED, ids=lambda f: f.__name__)
def test_inputs_keep_their_distances(fn, monkeypatch):
    seen = []

    def run(case, status=0, **kw):
        return [x for x in case.oracle()[:4]]

    def check(case, close=1e-9):
        seen.append(margins(case))
        return run(case)

    monkeypatch.setattr(gpu, "run", run)
    monkeypatch.setattr(gpu, "check", check)
    for kw in combinations(fn):
        fn(**kw)
    assert seen
    print(fn.__name__, len(seen), "cases, smallest test and draw over what they need:", *np.min(seen, 0))
    assert (np.min(seen, 0) > 1).all(), sorted(seen)[:5]
