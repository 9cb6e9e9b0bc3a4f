"""The oracle of the latent operators against hand-worked cases and against
each other: both forms of one attention, a step's slots and what append writes."""
import numpy as np

from oracle import latent_oracle as lo


def test_extend_by_hand():
    # Three sequences of a pool of 6 pages; page 4 and 1 held, 0 shared by nobody.
    table = np.array([[4, -1, -1], [1, -1, -1], [-1, -1, -1]], np.int32)
    ref = np.array([0, 1, 0, 0, 1, 0], np.int32)
    got = lo.extend(table, ref, np.array([15, 16, 0]), np.array([3, 1, 0]), 6)
    assert got[6] == 0
    assert got[0].tolist() == [[4, 0, -1], [1, 2, -1], [-1, -1, -1]]
    assert got[1].tolist() == [1, 1, 1, 0, 1, 0]
    assert got[2].tolist() == [0, 3, 4, 4]
    assert got[3].tolist() == [0, 0, 0, 1, -1, -1]
    assert got[4].tolist() == [15, 16, 17, 16, -1, -1]
    assert got[5].tolist() == [79, 0, 1, 32, -1, -1]


def test_extend_tree_positions():
    table, ref = np.full((1, 2), -1, np.int32), np.zeros(4, np.int32)
    got = lo.extend(table, ref, np.array([0]), np.array([5]), 5, np.array([1]), np.array([-1, 0, 0, 2, 1]))
    assert got[4].tolist() == [0, 1, 1, 2, 2] and got[5].tolist() == [0, 1, 2, 3, 4]


def test_extend_findings_change_nothing():
    table, ref = np.array([[0, -1], [1, -1]], np.int32), np.array([1, 2, 0], np.int32)
    for ctx, rows, most, bits in [([3, 16], [1, -1], 4, lo.BAD_ROWS), ([33, 16], [1, 1], 4, lo.CTX_OVERFLOW),
                                  ([3, 3], [1, 1], 4, lo.BAD_BLOCK), ([16, 16], [1, 1], 4, lo.NO_PAGES),
                                  ([3, 16], [2, 1], 2, lo.BAD_ROWS), ([17, 16], [1, 0], 4, lo.BAD_BLOCK)]:
        t, r, cu, seq, _, slot, bad = lo.extend(table, ref, np.array(ctx), np.array(rows), most)
        assert bad == bits and (t == table).all() and (r == ref).all() and not cu.any() and (slot == -1).all()


def test_rotations_agree():
    r = np.random.default_rng(0)
    x, a = r.standard_normal((3, 8)), r.standard_normal(4)
    one = lo.rotate(x, np.cos(a), np.sin(a), True)
    order = [0, 2, 4, 6, 1, 3, 5, 7]
    two = lo.rotate(x[:, order], np.cos(a), np.sin(a), False)
    assert np.allclose(one[:, order], two)
    z = (x[:, 0::2] + 1j * x[:, 1::2]) * np.exp(1j * a)
    assert np.allclose(one[:, 0::2], z.real) and np.allclose(one[:, 1::2], z.imag)


def test_both_forms_are_one_attention():
    """Absorbed queries over latents, then Wv, equal expanded keys and values."""
    r = np.random.default_rng(1)
    heads, nope, rope, latent, value, ctx, n = 3, 6, 4, 10, 5, 7, 4
    wk, wv = r.standard_normal((heads, nope, latent)), r.standard_normal((heads, value, latent))
    c, kr = r.standard_normal((ctx + n, latent)), r.standard_normal((ctx + n, rope))
    q = r.standard_normal((n, heads, nope + rope))
    absorbed = np.concatenate([np.einsum("nhd,hdl->nhl", q[..., :nope], wk), q[..., nope:]], 2)
    rows = np.concatenate([c, kr], 1)
    o, lse, _ = lo.latent(absorbed, lambda s, m: rows[:m], [0, n], [ctx], 0.3, latent)
    kv = np.concatenate([np.einsum("hdl,tl->thd", wk, c), np.einsum("hvl,tl->thv", wv, c)], 2)
    e, lse2, _ = lo.prompt(q, kv, kr, [0, n], [0, ctx + n], 0.3, nope)
    assert np.allclose(np.einsum("nhl,hvl->nhv", o, wv), e) and np.allclose(lse, lse2)


def test_rows_that_see_nothing():
    r = np.random.default_rng(2)
    q, kv, kr = r.standard_normal((5, 2, 8)), r.standard_normal((3, 2, 8)), r.standard_normal((3, 4))
    o, lse, _ = lo.prompt(q, kv, kr, [0, 5], [0, 3], 1.0, 4)
    assert (o[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()
    joined = np.logaddexp.reduce([lo.prompt(q[4:], kv[a:b], kr[a:b], [0, 1], [0, b - a], 1.0, 4, False)[1]
                                  for a, b in ((0, 2), (2, 3))])
    assert np.allclose(joined, lse[4:])
