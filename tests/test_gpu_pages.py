"""cache_fork, cache_free and cache_compact on the GPU against the plain forms, to the bit."""
import numpy as np
import pytest
import torch

from tests import pages_plain as plain
from tests.test_gpu_cache import _i32, _same

pytestmark = pytest.mark.gpu


class Pool:
    """R requests of the given lengths over a shuffled pool of N blocks; some share their first blocks with the one before."""

    def __init__(self, seq, bs, N, layers=1, heads=2, D=16, shared=None, seed=0, dtype=torch.bfloat16, order="tokens",
                 most=None):
        rng = np.random.default_rng(seed)
        self.rng, self.seq, self.bs, self.N = rng, np.array(seq, np.int32), bs, N
        R = len(seq)
        held = [-(-max(int(x), 0) // bs) for x in seq]
        self.most = (max(held) + 1) if most is None else most
        ids = rng.permutation(N).astype(np.int32)
        self.table, used = np.full((R, self.most), -7, np.int32), 0
        for r in range(R):
            first = 0 if shared is None else min(shared[r], held[r] if r == 0 else min(held[r], held[r - 1]))
            if first:
                self.table[r, :first] = self.table[r - 1, :first]
            self.table[r, first:held[r]] = ids[used:used + held[r] - first]
            used += held[r] - first
        assert used <= N
        self.free = np.full(N, -9, np.int32)
        self.free[: N - used] = ids[used:]
        self.count = N - used
        shape = (layers, N, bs, heads, D)
        g = torch.Generator(device="cuda").manual_seed(seed)
        perm = {"tokens": (0, 1, 2, 3, 4), "heads": (0, 1, 3, 2, 4), "layers": (1, 0, 2, 3, 4), "places": (2, 1, 0, 3, 4)}[order]
        back = [perm.index(i) for i in range(5)]
        self.k, self.v = (torch.randn([shape[i] for i in perm], generator=g, device="cuda").to(dtype).permute(back)
                          for _ in range(2))

    def host(self, t):
        return t.contiguous().view(torch.int16).cpu().numpy()

    def check_fork(self, sv, source, free=None, count=None):
        free, count = self.free if free is None else free, self.count if count is None else count
        source = np.array(source, np.int32)
        want = plain.fork(self.host(self.k), self.host(self.v), self.table, self.seq, source, free, count)
        table, dfree = _i32(self.table), _i32(free)
        for _ in range(2):  # again on the same inputs: the same
            got = sv.cache_fork(self.k, self.v, table, _i32(self.seq), _i32(source), dfree, _i32([count]))
            torch.cuda.synchronize()
            for name in ("status", "seq_len", "free_count"):
                _same(got[name], want[name], name)
            _same(table, want["block_table"], "block_table")
            np.testing.assert_array_equal(self.host(self.k), want["k"])
            np.testing.assert_array_equal(self.host(self.v), want["v"])
        _same(dfree, free, "free_blocks")
        return want

    def check_free(self, sv, leave, free=None, count=None):
        free, count = self.free if free is None else free, self.count if count is None else count
        leave = np.array(leave, np.int32)
        want = plain.free_rows(self.table, self.seq, leave, free, count, self.bs, self.N)
        table, dfree = _i32(self.table), _i32(free)
        for _ in range(2):
            got = sv.cache_free(table, _i32(self.seq), _i32(leave), dfree, _i32([count]), self.bs)
            torch.cuda.synchronize()
            for name in ("status", "seq_len", "free_count"):
                _same(got[name], want[name], name)
            _same(dfree, want["free_blocks"], "free_blocks")
        _same(table, self.table, "block_table")
        return want

    def check_compact(self, sv):
        want = plain.compact(self.host(self.k), self.host(self.v), self.table, self.seq)
        table = _i32(self.table)
        for _ in range(2):
            got = sv.cache_compact(self.k, self.v, table, _i32(self.seq))
            torch.cuda.synchronize()
            for name in ("status", "block_table", "free_blocks", "free_count"):
                _same(got[name], want[name], name)
            np.testing.assert_array_equal(self.host(self.k), want["k"])
            np.testing.assert_array_equal(self.host(self.v), want["v"])
        _same(table, self.table, "block_table")
        return want


# --- fork --------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("order", ["tokens", "heads", "layers", "places"])
@pytest.mark.parametrize("bs,layers,heads,D", [(8, 1, 1, 8), (16, 3, 2, 64), (24, 2, 3, 80), (128, 1, 4, 128)])
def test_fork(sv, bs, layers, heads, D, order):
    seq = [0, 1, bs - 1, bs, bs + 1, 3 * bs + 5, 0, 0, 0, 0, 0, 0, 0]
    p = Pool(seq, bs, 40, layers, heads, D, seed=bs, order=order)
    want = p.check_fork(sv, [-1, -1, -1, -1, -1, -1, 1, 2, 3, 4, 5, 5, 0])
    assert not want["status"].any() and want["seq_len"].tolist() == seq[:6] + [1, bs - 1, bs, bs + 1, 3 * bs + 5, 3 * bs + 5, 0]


def test_fork_many(sv):
    rng = np.random.default_rng(1)
    seq = np.concatenate([rng.integers(0, 200, 300), np.zeros(700, np.int64)])
    source = np.concatenate([np.full(300, -1), rng.integers(0, 300, 700)])
    both = rng.permutation(1000)  # rows and their sources in any order
    place = np.argsort(both)
    source = np.where(source >= 0, place[source], -1)[both]
    p = Pool(seq[both], 8, 9000, seed=2)
    p.check_fork(sv, source)


def test_forks_that_find_no_block(sv):
    seq = [20, 16, 0, 0, 0, 0, 0, 0]
    source = [-1, -1, 0, 1, 0, 1, 0, 1]
    for count in (0, 1, 2, 3, 4):
        p = Pool(seq, 8, 16, seed=count)
        want = p.check_fork(sv, source, count=count)
        assert (want["status"] == 256).sum() == max(0, 3 - count)
        assert want["seq_len"][[3, 5, 7]].tolist() == [16] * 3  # full blocks need none
    p = Pool(seq, 8, 16)
    p.check_fork(sv, source, count=-3), p.check_fork(sv, source, count=99, free=np.arange(16, dtype=np.int32)[::-1].copy())


def test_forks_that_are_none(sv):
    p = Pool([20, 9, 0, 0, 0, 0, 0], 8, 30, seed=3)
    p.seq[5] = -4
    want = p.check_fork(sv, [1, -1, 7, 2 ** 31 - 1, 4, 0, 5])
    # a row with tokens, no such rows, itself, a negative length, a source of one
    assert want["status"].tolist() == [16384, 0, 16384, 16384, 0, 1024 | 16384, 1024]
    p = Pool([20, 0, 0], 8, 30, seed=4, most=4)
    p.seq[0] = 33  # longer than its row
    assert p.check_fork(sv, [-1, 0, -1])["status"].tolist() == [1024, 1024, 0]
    p = Pool([20, 0, 12, 0], 8, 30, seed=5)
    p.table[0, 1], p.table[2, 1] = 30, -1  # a full block and a last one outside the pool
    assert p.check_fork(sv, [-1, 0, -1, 2])["status"].tolist() == [0, 2048, 0, 2048]
    p = Pool([20, 0], 8, 30, seed=6)
    p.free[p.count - 1] = 77  # the stack holds an id outside the pool
    assert p.check_fork(sv, [-1, 0])["status"].tolist() == [0, 2048]


def test_fork_in_a_long_cache(sv):
    """Offsets past 2^32 entries; only the blocks that matter are written."""
    N, bs, heads, D = 70000, 64, 8, 128
    k = torch.empty((1, N, bs, heads, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = _i32([[N - 1, N - 2], [-1, -1]])
    for c, x in ((k, 1.0), (v, 2.0)):
        c[0, N - 2] = x
        c[0, N - 3] = 0.0
    got = sv.cache_fork(k, v, table, _i32([bs + 9, 0]), _i32([-1, 0]), _i32(np.full(N, N - 3)), _i32([5]))
    assert got["free_count"].item() == 4 and table[1].tolist() == [N - 1, N - 3]
    for c, x in ((k, 1.0), (v, 2.0)):
        assert (c[0, N - 3, :9] == x).all() and (c[0, N - 3, 9:] == 0).all()
    # and the move of a compaction over the same distance
    got = sv.cache_compact(k, v, table, got["seq_len"])
    assert got["block_table"].tolist() == [[2, 1], [2, 0]] and got["free_count"].item() == N - 3
    for c, x in ((k, 1.0), (v, 2.0)):
        assert (c[0, 1] == x).all() and (c[0, 0, :9] == x).all() and (c[0, 0, 9:] == 0).all()


# --- free --------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("N", [1, 31, 32, 33, 300, 5000, 70001])
@pytest.mark.parametrize("R", [1, 2, 37, 300])
def test_free(sv, R, N):
    rng = np.random.default_rng(R * 7 + N)
    seq = rng.integers(0, max(1, 8 * N // R) + 1, R)
    seq[0] = min(8, 8 * N)
    while sum(-(-int(x) // 8) for x in seq) > N:
        seq //= 2
    shared = rng.integers(0, 4, R) * (np.arange(R) > 0)
    p = Pool(seq, 8, N, heads=1, D=8, shared=shared, seed=R)
    p.check_free(sv, rng.random(R) < 0.5)
    p.check_free(sv, np.ones(R)), p.check_free(sv, np.zeros(R)), p.check_free(sv, np.full(R, -2 ** 31))


def test_shared_blocks_stay_until_the_last_leaves(sv):
    p = Pool([40, 40, 40, 9], 8, 30, shared=[0, 3, 2, 0])  # 5 blocks, 2 more, 3 more
    assert p.check_free(sv, [1, 0, 0, 0])["free_count"][0] == p.count + 2
    assert p.check_free(sv, [1, 1, 0, 0])["free_count"][0] == p.count + 5
    assert p.check_free(sv, [1, 1, 1, 0])["free_count"][0] == p.count + 10


def test_blocks_are_pushed_once(sv):
    p = Pool([40, 17], 8, 20)
    p.table[0, 3] = p.table[0, 1]                  # the same block twice in a row
    p.free[p.count] = p.table[0, 2]                # one that is free already
    p.check_free(sv, [1, 0], count=p.count + 1)
    # a call whose lengths were not updated after the one before
    first = p.check_free(sv, [1, 0])
    again = p.check_free(sv, [1, 0], free=first["free_blocks"], count=first["free_count"][0])
    assert again["free_count"][0] == first["free_count"][0]


def test_free_with_bad_lengths_and_blocks(sv):
    p = Pool([30, 30, 30, 30, 30, 30], 8, 40, most=4)
    p.seq[:4] = -1, 33, -2 ** 31, 2 ** 31 - 1
    p.table[4, 1], p.table[5, 0] = 40, -1
    want = p.check_free(sv, [1, 1, 0, 0, 1, 0])
    assert want["status"].tolist() == [1024, 1024, 1024, 1024, 2048, 2048]
    p.free[0], p.free[1] = 99, -1                  # a stack with ids outside the pool
    p.check_free(sv, [0, 0, 0, 0, 1, 1]), p.check_free(sv, [0, 0, 0, 0, 1, 1], count=-7)
    p.check_free(sv, [1] * 6, count=1000)          # more than the stack holds: a full one


# the largest pool there may be, and those on both sides of where a thread block's shared memory holds all of its bits
@pytest.mark.parametrize("N", [812000, 828000, 1 << 22])
def test_free_the_largest_pools(sv, N):
    assert sv.MAX_BLOCKS == 1 << 22
    table = torch.arange(N, dtype=torch.int32, device="cuda").flip(0).view(4, N // 4).contiguous()
    free = torch.empty(N, dtype=torch.int32, device="cuda")
    got = sv.cache_free(table, _i32([N // 4 * 8] * 4), _i32([0, 1, 0, 1]), free, _i32([0]), 8)
    assert got["free_count"].item() == N // 2
    want = torch.cat([table[3].flip(0), table[1].flip(0)])
    assert torch.equal(free[: N // 2], want)
    with pytest.raises(sv.SpecVerifyError):
        sv.cache_free(table, _i32([8] * 4), _i32([0] * 4), torch.empty(sv.MAX_BLOCKS + 1, dtype=torch.int32, device="cuda"), _i32([0]), 8)


# --- compact -----------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("order", ["tokens", "heads", "layers", "places"])
@pytest.mark.parametrize("bs,layers,heads,D,N", [(8, 1, 1, 8, 40), (16, 3, 2, 64, 33), (24, 2, 3, 80, 100), (128, 1, 5, 128, 64),
                                                 (8, 1, 1, 16, 3000)])
def test_compact(sv, bs, layers, heads, D, N, order):
    rng = np.random.default_rng(N)
    seq = [0, 1, bs - 1, bs, bs + 1, 3 * bs + 5, 5 * bs]
    if N > 1000:
        seq += rng.integers(0, 30 * bs, 100).tolist()
    p = Pool(seq, bs, N, layers, heads, D, shared=[0] + [int(x) for x in rng.integers(0, 3, len(seq) - 1)], seed=bs, order=order)
    p.check_compact(sv)


def test_compact_full_empty_and_packed_pools(sv):
    Pool([80, 80], 8, 20).check_compact(sv)        # no gaps
    Pool([0, 0, 0], 8, 20).check_compact(sv)       # nothing held
    p = Pool([80, 33], 8, 40, layers=2)
    p.check_compact(sv)
    table = plain.compact(p.host(p.k), p.host(p.v), p.table, p.seq)["block_table"]
    p.table = table
    want = p.check_compact(sv)                     # packed already
    np.testing.assert_array_equal(want["block_table"], table)
    got = sv.cache_compact(p.k, p.v, torch.empty((0, 4), dtype=torch.int32, device="cuda"), _i32([]))
    assert got["free_count"].item() == 40 and got["free_blocks"].tolist() == list(range(39, -1, -1))
    one = Pool([3], 8, 1)
    one.check_compact(sv)


def test_compact_with_bad_lengths_and_blocks(sv):
    p = Pool([30, 30, 30, 30], 8, 40, most=4)
    p.seq[:2] = -1, 33
    p.table[2, 1], p.table[3, 0] = 40, -5
    assert p.check_compact(sv)["status"].tolist() == [1024, 1024, 2048, 2048]


@pytest.mark.parametrize("N", [1628000, 1648000, 1 << 22])
def test_compact_the_largest_pools(sv, N):
    k = torch.zeros((N, 8, 1, 8), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.arange(N - 1, N - 2049, -1, dtype=torch.int32, device="cuda").view(8, 256)
    k[N - 2048:, 0, 0, 0] = torch.arange(2048, device="cuda").bfloat16()
    got = sv.cache_compact(k, v, table.contiguous(), _i32([2048] * 8))
    assert got["free_count"].item() == N - 2048
    assert torch.equal(got["block_table"], table - (N - 2048))
    assert torch.equal(k[:2048, 0, 0, 0], k[N - 2048:, 0, 0, 0])
    assert torch.equal(got["free_blocks"][: N - 2048], torch.arange(N - 1, 2047, -1, dtype=torch.int32, device="cuda"))


# --- all three ---------------------------------------------------------------------------------------------------
def test_captured_and_replayed(sv):
    p = Pool([40, 23, 0, 9], 8, 30, layers=2)
    table, seq, free, count = _i32(p.table), _i32(p.seq), _i32(p.free), _i32([p.count])
    source, leave = _i32([-1, -1, 1, -1]), _i32([1, 0, 0, 0])
    calls = [lambda: sv.cache_fork(p.k, p.v, table, seq, source, free, count),
             lambda: sv.cache_free(table, seq, leave, free, count, 8), lambda: sv.cache_compact(p.k, p.v, table, seq)]
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = call()
        for t in got.values():
            t.fill_(-3)
        g.replay(), g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[name], want[name]) for name in want)


def test_layer_by_layer(sv):
    """A call for each layer on the same inputs does what one call does for all of them."""
    p = Pool([40, 23, 0, 9], 8, 30, layers=3)
    table, seq, free, count, source = _i32(p.table), _i32(p.seq), _i32(p.free), _i32([p.count]), _i32([-1, -1, 1, -1])
    k, v = [x.clone() for x in p.k], [x.clone() for x in p.v]
    one = sv.cache_fork(p.k, p.v, table, seq, source, free, count)
    forked = table.clone()
    for layer in range(3):
        each = sv.cache_fork(k[layer], v[layer], table, seq, source, free, count)
        assert torch.equal(table, forked) and all(torch.equal(each[name], one[name]) for name in one)
    seq_len = one["seq_len"]
    one = sv.cache_compact(p.k, p.v, table, seq_len)
    for layer in range(3):
        each = sv.cache_compact(k[layer], v[layer], table, seq_len)
        assert all(torch.equal(each[name], one[name]) for name in one)
        assert torch.equal(k[layer], p.k[layer]) and torch.equal(v[layer], p.v[layer])


def test_a_replayed_graph_takes_new_tables(sv):
    """The lengths, tables and the stack of a captured call may change between its replays."""
    p, q = (Pool([40, 23, 0, 9, x, 0], 8, 60, layers=2, seed=x, most=9) for x in (17, 64))
    table, seq, free, count = _i32(p.table), _i32(p.seq), _i32(p.free), _i32([p.count])
    source, leave = _i32([-1, -1, 1, -1, -1, 0]), _i32([1, 0, 0, 1, 0, 0])
    graphs, outs = [], []
    for call in (lambda: sv.cache_fork(p.k, p.v, table, seq, source, free, count),
                 lambda: sv.cache_free(table, seq, leave, free, count, 8), lambda: sv.cache_compact(p.k, p.v, table, seq)):
        call()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call())
    new_source, new_leave = [-1, -1, 4, -1, -1, 2], [0, 1, 0, 0, 1, 0]
    wants = [plain.fork(q.host(q.k), q.host(q.v), q.table, q.seq, new_source, q.free, q.count),
             plain.free_rows(q.table, q.seq, np.array(new_leave), q.free, q.count, 8, 60),
             plain.compact(q.host(q.k), q.host(q.v), q.table, q.seq)]
    for g, got, want in zip(graphs, outs, wants):
        for mine, other in ((table, q.table), (seq, q.seq), (free, q.free), (count, [q.count]), (source, new_source),
                            (leave, new_leave)):
            mine.copy_(_i32(other))
        p.k.copy_(q.k), p.v.copy_(q.v)
        g.replay()
        torch.cuda.synchronize()
        for name in got:
            _same(got[name], want[name], name)
        if "k" in want:
            np.testing.assert_array_equal(p.host(p.k), want["k"])
            np.testing.assert_array_equal(p.host(p.v), want["v"])


def test_two_streams_at_once(sv):
    """Calls that share nothing, side by side."""
    pools = [Pool(np.random.default_rng(i).integers(0, 900, 50), 8, 6000, layers=2, seed=i) for i in range(2)]
    wants = [plain.compact(p.host(p.k), p.host(p.v), p.table, p.seq) for p in pools]
    args = [(_i32(p.table), _i32(p.seq)) for p in pools]
    streams = [torch.cuda.Stream() for _ in pools]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [sv.cache_compact(p.k, p.v, *a, stream=s) for p, a, s in zip(pools, args, streams)]
    torch.cuda.synchronize()
    for p, g, w in zip(pools, got, wants):
        _same(g["block_table"], w["block_table"], "block_table")
        np.testing.assert_array_equal(p.host(p.k), w["k"])


def test_outputs_over_inputs_are_refused(sv):
    p = Pool([40, 0], 8, 30)
    table, seq, free, count = _i32(p.table), _i32(p.seq), _i32(p.free), _i32([p.count])
    two, other = _i32([-1, 0]), _i32([0, 0])
    for out in (dict(seq_len=seq, free_count=_i32([0])), dict(seq_len=two, free_count=_i32([0])),
                dict(seq_len=other, free_count=count)):
        with pytest.raises(sv.SpecVerifyError):
            sv.cache_fork(p.k, p.v, table, seq, two, free, count, out=out)
        with pytest.raises(sv.SpecVerifyError):
            sv.cache_free(table, seq, two, free, count, 8, out=out)


def test_no_requests(sv):
    none, table = _i32([]), torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    p = Pool([3], 8, 10)
    assert sv.cache_fork(p.k, p.v, table, none, none, _i32(range(10)), _i32([7]))["free_count"].item() == 7
    assert sv.cache_free(table, none, none, _i32(range(10)), _i32([7]), 8)["free_count"].item() == 7


def test_refusals(sv):
    p = Pool([40, 0], 8, 30, layers=2)
    table, seq, free, count = _i32(p.table), _i32(p.seq), _i32(p.free), _i32([p.count])
    two, i32 = _i32([-1, 0]), torch.int32
    calls = dict(fork=lambda table=table, seq=seq, two=two, free=free, count=count, k=p.k, **kw:
                 sv.cache_fork(k, p.v, table, seq, two, free, count, **kw),
                 free=lambda table=table, seq=seq, two=two, free=free, count=count, **kw:
                 sv.cache_free(table, seq, two, free, count, 8, **kw),
                 compact=lambda table=table, seq=seq, k=p.k, **kw: sv.cache_compact(k, p.v, table, seq, **kw))
    for name, call in calls.items():
        out = call()
        for bad in (table[:1], table.flatten(), table.long(), table.cpu(), table.t().contiguous().t()):
            with pytest.raises(ValueError):
                call(table=bad)
        with pytest.raises(ValueError):
            call(seq=seq.long())
        if name != "compact":
            for bad in (two[:1], two.float(), two.cpu()):
                with pytest.raises(ValueError):
                    call(two=bad)
            with pytest.raises(ValueError):
                call(count=_i32([1, 2]))
            with pytest.raises(ValueError):
                call(free=free.cpu())
        if name != "free":
            with pytest.raises(ValueError):
                call(k=p.k[:, :29])
            with pytest.raises(TypeError):
                call(k=p.k.half())
        for key, t in out.items():
            for bad in (t.reshape(-1)[:-1].clone(), t.cpu(), t.double()):
                with pytest.raises(ValueError, match=key):
                    call(out=dict(out, **{key: bad}))
        call(out={key: t for key, t in out.items() if key != "status"})
    with pytest.raises(ValueError, match="free_blocks"):
        calls["fork"](free=free[:29].contiguous())
    with pytest.raises(sv.SpecVerifyError):
        calls["compact"](workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="workspace"):
        calls["compact"](workspace=torch.empty(4096, dtype=torch.uint8))
    with pytest.raises(sv.SpecVerifyError):  # tables in place
        calls["compact"](out=dict(block_table=table, free_blocks=torch.empty(30, dtype=i32, device="cuda"),
                                  free_count=torch.empty(1, dtype=i32, device="cuda")))
    torch.cuda.synchronize()
