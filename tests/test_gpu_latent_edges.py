"""Edges of attention over a latent cache: queries and cached values that are no
numbers where a sequence has one tile or every tile moves a row's maximum, and
rows in the company of other sequences (GB300)."""
import pytest

from latent_util import Latent

import speculative_decoding_verify_kv_gb300 as va

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def rising(case, upto):
    """Column 0 of sequence 0's first tokens grows with the token."""
    t = torch.arange(upto, device="cuda")
    table = case.kv.block_table[0].long()
    case.kv.cache[table[t // 16], t % 16, 0] = (t.float() / 6).to(case.kv.cache.dtype)


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("heads,rows", [(2, 5), (16, 1), (6, 5), (32, 1), (40, 2)])
@pytest.mark.parametrize("ctx", [0, 1, 40, 59, 130])
@pytest.mark.parametrize("splits", [1, 3])
def test_nan_query_of_few_tokens(latent, heads, rows, ctx, splits):
    """One tile or a few: the row is NaN, not an empty row's outputs."""
    case = Latent("bf16", heads, latent, [ctx, 7], [rows, 1], seed=ctx + heads, splits=splits)
    want = [t.clone() for t in case.run()]
    case.q[rows - 1, 1, 7] = float("nan")
    o, lse = case.run()
    assert case.status.item() == 0
    assert o[rows - 1, 1].isnan().all() and lse[rows - 1, 1].isnan()
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[rows - 1, 1] = False
    assert torch.equal(o[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("heads", [4, 20, 48])
@pytest.mark.parametrize("splits", [1, 4])
def test_nan_query_of_rising_scores(latent, heads, splits):
    """Every tile, the last one too, moves the other rows' maximum."""
    case = Latent("bf16", heads, latent, [895], [1], seed=4, splits=splits, scale=0.1)
    case.q.zero_()
    case.q[..., 0] = 8.0
    rising(case, 896)
    case.q[0, 2, 5] = float("nan")
    o, lse = case.run()
    assert o[0, 2].isnan().all() and lse[0, 2].isnan()
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[0, 2] = False
    assert o[keep].isfinite().all() and lse[keep].isfinite().all()


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("heads", [3, 24, 40])
@pytest.mark.parametrize("token", [0, 37, 130])
def test_nan_token(latent, heads, token):
    """A cached key that every row sees and that is no number makes them NaN."""
    case = Latent("bf16", heads, latent, [140], [1], seed=heads, splits=1)
    case.kv.cache[case.kv.block_table[0, token // 16].long(), token % 16, latent + 3] = float("nan")
    o, lse = case.run()
    assert o.isnan().all() and lse.isnan().all()
