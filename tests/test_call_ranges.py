"""Numbers that do not fit the C structs are refused, not cut to 32 bits
(2^32 + 5 tokens of window would be 5).  No GPU."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verify_kv_gb300 as va
from test_call_streams import arguments, z


@pytest.mark.parametrize("kw", [dict(window=2 ** 32 + 5), dict(window=2 ** 31), dict(window=8, sinks=2 ** 32),
                                dict(window=8, sinks=-2 ** 32 + 1)])
def test_windows(kw):
    _, (p, kv, mode, _), _ = arguments()["window"]
    with pytest.raises(ValueError, match="32 bits"):
        va.WindowCall(p, kv, mode, va.Window(**kw))
    with pytest.raises(ValueError, match="32 bits"):
        va.window_splits(p, kv, va.Window(**kw))
    va.WindowCall(p, kv, mode, va.Window(2 ** 31 - 1, 2 ** 31 - 1))


def test_vocabularies():
    _, (p, draft, mode), _ = arguments()["accept"]
    draft.logits_stride, draft.vocab = 10, 2 ** 32 + 10
    with pytest.raises(ValueError):
        va.AcceptCall(p, draft, mode)
    with pytest.raises(ValueError, match="32 bits"):
        draft.c()


class Large(torch.Tensor):
    """A tensor that says it has more elements than it has."""
    def numel(self):
        return 2 ** 32 + 8


def test_pools():
    large = z(8).as_subclass(Large)
    with pytest.raises(ValueError, match="32 bits"):
        va.PagePool(z(2, 4), large).c()
    with pytest.raises(ValueError, match="32 bits"):
        va.CompactCall(va.PagePool(z(2, 4), large))
    with pytest.raises(ValueError, match="32 bits"):
        va.ForkCall(va.PagePool(z(2, 4), z(16)), large, large, large, large)
    with pytest.raises(ValueError, match="32 bits"):
        va.PageCopyCall([z(4, 8)], z(1, 2).as_subclass(Large), z(1))
