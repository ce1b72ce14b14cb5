"""Page calls whose outputs share bytes with inputs are refused; nothing here touches a GPU."""
from tests.test_cache_abi import BUF, P, _cache, m  # noqa: F401

A, B, C, D, E, F, G, WS = (P(0x100000 + 0x10000 * i) for i in range(8))  # arrays that are 64 KB apart
R, MB, NB = 6, 5, 40


def _fork(m, table=A, seq=B, source=C, free=D, count=E, seq_out=F, count_out=G, status=None):  # noqa: F811
    return m.load().sv_cache_fork(_cache(m, num_blocks=NB), table, MB, seq, R, source, free, count, seq_out, count_out, status,
                                  None)


def _free(m, table=A, seq=B, leave=C, free=D, count=E, seq_out=F, count_out=G, status=None):  # noqa: F811
    return m.load().sv_cache_free(table, MB, seq, leave, R, 16, free, count, NB, seq_out, count_out, status, None)


def _compact(m, table=A, seq=B, out=C, free=D, count=E, status=None, ws=WS):  # noqa: F811
    return m.load().sv_cache_compact(_cache(m, num_blocks=NB), table, MB, seq, R, out, free, count, status, ws, 1 << 16, None)


def _last(array, entries):
    """The last entry of an array."""
    return P(array.value + 4 * (entries - 1))


def _before(array, entries):
    """An array of so many entries whose last one is the first one of `array`."""
    return P(array.value - 4 * (entries - 1))


def test_outputs_over_inputs(m):  # noqa: F811
    sizes = dict(table=R * MB, seq=R, free=NB, count=1)
    for call, two in ((_fork, "source"), (_free, "leave")):
        arrays = dict(zip(("table", "seq", two, "free", "count"), (A, B, C, D, E)))
        for name, array in arrays.items():
            n = sizes.get(name, R)
            for out, entries in (("status", R), ("seq_out", R), ("count_out", 1)):
                for bad in (array, _last(array, n), _before(array, entries)):
                    assert call(m, **{out: bad}) == -1, (call, name, out)
    for array, n in ((A, R * MB), (B, R)):
        for out, entries in (("status", R), ("out", R * MB)):
            for bad in (array, _last(array, n), _before(array, entries)):
                assert _compact(m, **{out: bad}) == -1, (n, out)
        assert _compact(m, ws=array) == -1


def test_arrays_side_by_side(m):  # noqa: F811
    import torch

    if torch.cuda.is_available():
        return  # these calls are valid
    for call in (_fork, _free):
        assert call(m) == call(m, status=P(0x200000)) == -8
        assert call(m, seq_out=P(B.value + 4 * R), count_out=P(D.value + 4 * NB), status=P(A.value + 4 * R * MB)) == -8
        assert call(m, seq_out=P(B.value - 4 * R), count_out=P(D.value - 4), status=P(A.value - 4 * R)) == -8
    assert _compact(m) == _compact(m, status=P(B.value + 4 * R), out=P(A.value + 4 * R * MB)) == -8
