"""What replayed page calls write in place, and forks whose thread blocks take several shares of a last block."""
import numpy as np
import pytest
import torch

from tests import pages_plain as plain
from tests.test_gpu_cache import _i32, _same
from tests.test_gpu_pages import Pool

pytestmark = pytest.mark.gpu


def _calls(sv, p, table, seq, free, count, source, leave):
    return dict(fork=lambda: sv.cache_fork(p.k, p.v, table, seq, source, free, count),
                free=lambda: sv.cache_free(table, seq, leave, free, count, p.bs),
                compact=lambda: sv.cache_compact(p.k, p.v, table, seq))


def _want(which, p, source, leave):
    if which == "fork":
        return plain.fork(p.host(p.k), p.host(p.v), p.table, p.seq, source, p.free, p.count)
    if which == "free":
        return plain.free_rows(p.table, p.seq, np.array(leave), p.free, p.count, p.bs, p.N)
    return plain.compact(p.host(p.k), p.host(p.v), p.table, p.seq)


@pytest.mark.parametrize("which", ["fork", "free", "compact"])
def test_a_replay_writes_in_place(sv, which):
    """Captured over one pool, replayed twice each over two others: tables, stack and caches are what the formula gives."""
    p, *others = (Pool([40, 23, 0, 9, x, 0, 0], 8, 60, layers=2, seed=x, most=9) for x in (17, 64, 31))
    source, leave = [-1, -1, 1, -1, -1, 0, -1], [1, 0, 0, 1, 0, 0, 0]
    d = dict(table=_i32(p.table), seq=_i32(p.seq), free=_i32(p.free), count=_i32([p.count]), source=_i32(source),
             leave=_i32(leave))
    call = _calls(sv, p, **d)[which]
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    for q in others:
        source, leave = [-1, -1, 4, -1, -1, 1, 4], [0, 1, 0, 0, 1, 0, 0]
        want = _want(which, q, source, leave)
        k, v = q.k.clone(), q.v.clone()
        for _ in range(2):
            for t in got.values():
                t.fill_(-3)
            for name, x in dict(table=q.table, seq=q.seq, free=q.free, count=[q.count], source=source, leave=leave).items():
                d[name].copy_(_i32(x))
            p.k.copy_(k), p.v.copy_(v)
            g.replay()
            torch.cuda.synchronize()
            for name in got:
                _same(got[name], want[name], name)
            _same(d["table"], want["block_table"] if which == "fork" else q.table, "block_table")
            _same(d["free"], want["free_blocks"] if which == "free" else q.free, "free_blocks")
            for name, x in dict(seq=q.seq, count=[q.count], source=source, leave=leave).items():
                _same(d[name], np.array(x, np.int32), name)
            np.testing.assert_array_equal(p.host(p.k), want.get("k", p.host(k)))
            np.testing.assert_array_equal(p.host(p.v), want.get("v", p.host(v)))


@pytest.mark.parametrize("R,bs,layers,heads,D", [(1000, 128, 1, 2, 16), (3000, 64, 1, 1, 8), (1100, 128, 3, 8, 64),
                                                 (9800, 24, 1, 1, 8)])
@pytest.mark.parametrize("order", ["tokens", "heads"])
def test_forks_of_large_tables(sv, R, bs, layers, heads, D, order):
    """So many rows that a thread block takes several of a last block's shares, of eight tokens each."""
    columns = -(-2 * layers * heads * (D // 8) // 128)
    assert 64 * torch.cuda.get_device_properties(0).multi_processor_count // (R * columns) < -(-bs // 8)
    lengths = [1, 7, 8, 9, bs // 2, bs - 1, bs, bs + 1, 2 * bs - 7, 2 * bs + bs // 2 + 3]
    seq, source = np.zeros(R, np.int64), np.full(R, -1)
    at = np.linspace(0, R - 40, len(lengths)).astype(int)
    seq[at] = lengths
    source[at + 3], source[at + 17], source[R - 1] = at, at[::-1], at[-1]
    p = Pool(seq, bs, 70, layers, heads, D, seed=bs, order=order)
    want = p.check_fork(sv, source)
    assert not want["status"].any() and (want["seq_len"] > 0).sum() == 3 * len(lengths) + 1
