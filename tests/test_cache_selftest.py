"""Argument checks of the attention call's self-test; nothing here touches a GPU."""
import torch

from tests.test_cache_abi import BUF, WS, _cache, _heads, m  # noqa: F401


def test_the_stop_checks_its_arguments_as_the_call_does(m):  # noqa: F811
    f = m.load().sv_selftest_tree_attention_stop

    def call(cta=0, cache=None, R=1, ws=WS):
        q = _heads(m)
        return f(q, cache or _cache(m), BUF, 4, BUF, BUF, R, 3, None, 0, 1.0, q, None, None, ws, 1 << 40, cta, None)

    assert call(cta=-1) == -1
    assert call(R=-1) == -1 and call(R=0) == 0
    assert call(cache=_cache(m, dtype=1)) == -2 and call(ws=None) == -6
    if not torch.cuda.is_available():
        assert call() == -8
