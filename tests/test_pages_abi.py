"""Argument checks of the operators at the two ends of a verify step; nothing here touches a GPU."""
import ctypes as C

import pytest

from tests.test_cache_abi import BUF, WS, P, _cache, _heads, m  # noqa: F401

ODD, MISALIGNED, OUT = P(0x10002), P(0x10001), P(0x30000)


def _rows(m, width=64, dtype=0, data=0x10000, stride=None):  # noqa: F811
    return m.SvRows(data, dtype, width, width if stride is None else stride)


def test_rules_have_the_layout_of_the_header(m):  # noqa: F811
    want = [("history", 0), ("history_len", 8), ("prompt_len", 16), ("history_width", 24), ("repetition", 32),
            ("presence", 40), ("frequency", 48), ("bias_start", 56), ("bias_id", 64), ("bias_value", 72),
            ("bias_entries", 80), ("mask", 88), ("masks", 96), ("mask_words", 100), ("mask_row", 104)]
    assert [(n, getattr(m.SvLogitRules, n).offset) for n, _ in m.SvLogitRules._fields_] == want
    assert C.sizeof(m.SvLogitRules) == 112


def test_adjust_checks(m):  # noqa: F811
    f = m.load().sv_adjust_logits

    def call(R=2, k=3, branches=2, draft=BUF, rows=None, out=None, status=None, **rules):
        rows = rows or _rows(m)
        return f(rows, R, k, branches, draft, m.SvLogitRules(**rules), out or rows, status, None)

    assert call(R=0) == 0
    assert call(R=-1) == -1 and call(k=-1) == -1 and call(branches=0) == -1 and call(k=0) == -1
    assert call(k=257) == -4 and call(branches=9) == -4
    assert call(draft=None) == -1 and call(draft=ODD) == -7
    assert call(rows=_rows(m, dtype=2)) == -2 and call(out=_rows(m, dtype=1)) == -2
    assert call(out=_rows(m, width=32, stride=64)) == -3 and call(rows=_rows(m, width=0)) == -3
    assert call(rows=_rows(m, stride=32)) == -3 and call(rows=_rows(m, data=None)) == -1
    assert call(rows=_rows(m, data=0x10001)) == -7
    assert call(out=_rows(m, stride=128)) == -3                      # in place, but not row by row
    # 14 rows of 64 entries of 2 bytes: the other matrix may be the columns beside them, and nothing that meets them
    wide = lambda data: _rows(m, data=data, stride=128)  # noqa: E731
    for data in (0x10000 + 2, 0x10000 + 126, 0x10000 + 256 + 130, 0x10000 - 256 * 13 - 126):
        assert call(rows=wide(0x10000), out=wide(data)) == -1, data
    assert call(rows=wide(0x10000), out=_rows(m, data=0x10000 + 128)) == -1
    assert call(R=1, k=0, branches=1, out=_rows(m, data=0x10000 + 126)) == -1
    assert call(history=BUF.value, history_width=8) == -1            # no lengths
    assert call(history=BUF.value, history_len=BUF.value, history_width=-1) == -1
    assert call(history=BUF.value, history_len=BUF.value, history_width=524288) == -4
    for name in ("history", "history_len", "prompt_len"):
        assert call(**dict(dict(history=BUF.value, history_len=BUF.value, history_width=8), **{name: ODD.value})) == -7
    for name in ("repetition", "presence", "frequency"):
        assert call(**{name: ODD.value}) == -7
    bias = dict(bias_start=BUF.value, bias_id=BUF.value, bias_value=BUF.value, bias_entries=4)
    for name in ("bias_start", "bias_id", "bias_value"):
        assert call(**dict(bias, **{name: None})) == -1 and call(**dict(bias, **{name: ODD.value})) == -7
    assert call(**dict(bias, bias_entries=-1)) == -1
    mask = dict(mask=BUF.value, masks=5, mask_words=2, mask_row=BUF.value)
    assert call(**dict(mask, mask_words=1)) == -3                    # narrower than the rows
    assert call(**dict(mask, mask_row=None)) == -3                   # 14 rows, 5 masks
    assert call(mask_row=BUF.value) == -1                            # no masks
    assert call(**dict(mask, masks=-1)) == -1 and call(**dict(mask, mask_words=-1)) == -1
    assert call(**dict(mask, mask=ODD.value)) == -7 and call(**dict(mask, mask_row=ODD.value)) == -7
    assert call(status=ODD) == -7


def test_norm_rope_checks(m):  # noqa: F811
    f = m.load().sv_norm_rope_cache

    def call(q=None, k=None, rot=64, cache=None, qw=BUF, kw=BUF, dtype=1, eps=1e-6, pos=BUF, out=None, inter=0):
        q, k = q or _heads(m), k or _heads(m, heads=2)
        return f(q, k, k, pos, BUF, BUF, rot, inter, 1.0, qw, kw, dtype, eps, out or q, cache or _cache(m), None)

    assert call(q=_heads(m, tokens=0), k=_heads(m, heads=2, tokens=0)) == 0
    assert call(eps=-1e-6) == -1 and call(eps=float("nan")) == -1 and call(eps=float("inf")) == -1
    assert call(dtype=2) == -2 and call(dtype=3) == -2               # fp16 weights beside bf16 heads
    assert call(qw=ODD) == -7 and call(kw=ODD) == -7 and call(dtype=0, kw=MISALIGNED) == -7
    assert call(rot=66) == -3 and call(inter=2) == -1 and call(pos=None) == -1
    assert call(k=_heads(m, heads=3)) == -3 and call(out=_heads(m, dtype=2)) == -2
    assert call(cache=_cache(m, layers=2)) == -3


def test_fork_checks(m):  # noqa: F811
    f = m.load().sv_cache_fork

    def call(R=2, mb=4, cache=None, table=BUF, seq=BUF, source=BUF, free=BUF, count=BUF, seq_out=OUT, count_out=OUT,
             status=None):
        return f(cache or _cache(m), table, mb, seq, R, source, free, count, seq_out, count_out, status, None)

    assert call(R=0) == 0
    assert call(R=-1) == -1 and call(mb=-1) == -1 and call(mb=1 << 28) == -4
    assert call(cache=_cache(m, layers=600000)) == -4 and call(cache=_cache(m, dtype=1)) == -2
    assert call(seq_out=BUF) == -1 and call(count_out=BUF) == -1     # in place
    for name in ("table", "seq", "source", "free", "count", "seq_out", "count_out"):
        assert call(**{name: None}) == -1 and call(**{name: ODD}) == -7
    assert call(status=ODD) == -7


def test_free_checks(m):  # noqa: F811
    f = m.load().sv_cache_free

    def call(R=2, bs=16, mb=4, nb=8, table=BUF, seq=BUF, leave=BUF, free=BUF, count=BUF, seq_out=OUT, count_out=OUT,
             status=None):
        return f(table, mb, seq, leave, R, bs, free, count, nb, seq_out, count_out, status, None)

    assert call(R=0) == 0
    assert call(R=-1) == -1 and call(mb=-1) == -1 and call(bs=0) == -1 and call(nb=-1) == -1
    assert call(mb=1 << 28) == -4 and call(nb=(1 << 22) + 1) == -4
    assert call(seq_out=BUF) == -1 and call(count_out=BUF) == -1     # in place
    for name in ("table", "seq", "leave", "free", "count", "seq_out", "count_out"):
        assert call(**{name: None}) == -1 and call(**{name: ODD}) == -7
    assert call(status=ODD) == -7


def test_compact_checks(m):  # noqa: F811
    lib = m.load()
    f = lib.sv_cache_compact

    def call(R=2, mb=4, cache=None, table=BUF, seq=BUF, out=P(0x30000), free=BUF, count=BUF, status=None, ws=WS,
             nbytes=1 << 30):
        return f(cache or _cache(m), table, mb, seq, R, out, free, count, status, ws, nbytes, None)

    assert call(R=-1) == -1 and call(mb=-1) == -1 and call(mb=1 << 28) == -4
    assert call(cache=_cache(m, num_blocks=(1 << 22) + 1)) == -4 and call(cache=_cache(m, k=None)) == -1
    assert call(out=BUF) == -1                                       # the table itself
    for name in ("table", "seq", "out", "free", "count"):
        assert call(**{name: None}) == -1 and call(**{name: ODD}) == -7
    assert call(status=ODD) == -7
    assert call(ws=None) == -6 and call(nbytes=8) == -6 and call(ws=P(0x20010)) == -6
    size = lib.sv_cache_compact_workspace
    assert size(0) == 0 and size((1 << 22) + 1) == 0 and size(4) >= 48 and size(1 << 22) > 0


def test_valid_calls_without_a_device(m):  # noqa: F811
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    lib = m.load()
    q, k, rows = _heads(m), _heads(m, heads=2), _rows(m)
    assert lib.sv_adjust_logits(rows, 2, 3, 2, BUF, m.SvLogitRules(), rows, None, None) == -8
    wide = lambda data: _rows(m, data=data, stride=128)  # noqa: E731
    for data in (0x10000 + 128, 0x10000 - 128, 0x10000 + 256 * 14, 0x10000 - 256 * 14, 0x10000 + 256 * 5 + 128):
        assert lib.sv_adjust_logits(wide(0x10000), 2, 3, 2, BUF, m.SvLogitRules(), wide(data), None, None) == -8, data
    assert lib.sv_norm_rope_cache(q, k, k, BUF, BUF, BUF, 64, 0, 1.0, None, None, 7, 1e-6, q, _cache(m), None) == -8
    assert lib.sv_cache_fork(_cache(m), BUF, 4, BUF, 2, BUF, BUF, BUF, OUT, OUT, None, None) == -8
    assert lib.sv_cache_free(BUF, 4, BUF, BUF, 2, 16, BUF, BUF, 8, OUT, OUT, None, None) == -8
    assert lib.sv_cache_compact(_cache(m), BUF, 4, BUF, 2, P(0x30000), BUF, BUF, None, WS, 1 << 20, None) == -8
