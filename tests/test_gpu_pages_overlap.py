"""Page calls whose arrays share bytes are refused, and leave everything as it was."""
import pytest
import torch

from tests.test_gpu_cache import _i32
from tests.test_gpu_pages import Pool

pytestmark = pytest.mark.gpu


def _setup():
    p = Pool([40, 0, 23], 8, 30, layers=2)
    t = dict(table=_i32(p.table), seq=_i32(p.seq), free=_i32(p.free), count=_i32([p.count]), source=_i32([-1, 0, -1]),
             leave=_i32([1, 0, 0]))
    return p, t


def _refused(sv, p, tensors, call):
    before = [t.clone() for t in (p.k, p.v, *tensors)]
    with pytest.raises(sv.SpecVerifyError, match="-1"):
        call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (p.k, p.v, *tensors)))


def _room(*like):
    return [torch.full_like(t, -5) for t in like]


@pytest.mark.parametrize("which", ["fork", "free"])
def test_fork_and_free(sv, which):
    p, t = _setup()
    two = t["source" if which == "fork" else "leave"]

    def call(out, table=t["table"], seq=t["seq"], two=two, free=t["free"], count=t["count"]):
        if which == "fork":
            return sv.cache_fork(p.k, p.v, table, seq, two, free, count, out=out)
        return sv.cache_free(table, seq, two, free, count, 8, out=out)

    def fresh():
        seq, count, status = _room(t["seq"], t["count"], t["seq"])
        return dict(seq_len=seq, free_count=count, status=status)

    inputs = [t["table"], t["seq"], two, t["free"], t["count"]]
    for name in ("seq_len", "free_count", "status"):
        for x in inputs:
            n = 1 if name == "free_count" else 3
            flat = x.view(-1)
            for bad in ([flat[-n:]] if len(flat) >= n else []) + [flat]:
                if bad.numel() >= n:
                    _refused(sv, p, inputs, lambda: call(dict(fresh(), **{name: bad})))
    # outputs that share bytes
    room = torch.full((8,), -5, dtype=torch.int32, device="cuda")
    for out in (dict(seq_len=room[:3], status=room[:3]), dict(seq_len=room[:3], status=room[2:5]),
                dict(seq_len=room[:3], free_count=room[2:3]), dict(status=room[:3], free_count=room[1:2])):
        _refused(sv, p, [*inputs, room], lambda: call(dict(fresh(), **out)))
    # what is written in place over what is read
    n = t["free"].numel()
    arena = torch.full((n + 3,), 1, dtype=torch.int32, device="cuda")
    if which == "fork":
        over = dict(table=torch.zeros((3, 6), dtype=torch.int32, device="cuda"))
        pairs = [dict(over, seq=over["table"].view(-1)[3:6]), dict(over, two=over["table"].view(-1)[15:]),
                 dict(over, count=over["table"].view(-1)[:1]), dict(table=arena[:18].view(3, 6), free=arena[:n])]
    else:
        pairs = [dict(free=arena[:n], table=arena[n - 3:].view(3, 2)), dict(free=arena[:n], seq=arena[n - 1:n + 2]),
                 dict(free=arena[:n], two=arena[n - 1:n + 2]), dict(free=arena[:n], count=arena[7:8])]
    for pair in pairs:
        _refused(sv, p, [*inputs, *pair.values()], lambda: call(fresh(), **pair))
    # side by side in one allocation: taken
    call(dict(seq_len=room[:3], free_count=room[3:4], status=room[4:7]))
    torch.cuda.synchronize()
    assert room[7].item() == -5 and room[3].item() >= 0 and not room[4:7].any()


def test_compact(sv):
    p, t = _setup()
    R, most = t["table"].shape
    N = t["free"].numel()

    def fresh():
        table, free, count, status = _room(t["table"], t["free"], t["count"], t["seq"])
        return dict(block_table=table, free_blocks=free, free_count=count, status=status)

    inputs = [t["table"], t["seq"]]
    call = lambda out, ws=None, table=t["table"], seq=t["seq"]: sv.cache_compact(p.k, p.v, table, seq, out=out, workspace=ws)  # noqa: E731
    flat = t["table"].view(-1)
    for bad in (dict(status=t["seq"]), dict(status=flat[:3]), dict(status=flat[-3:]), dict(free_count=t["seq"][2:]),
                dict(free_count=flat[-1:]), dict(block_table=t["table"])):
        _refused(sv, p, inputs, lambda: call(dict(fresh(), **bad)))
    arena = torch.zeros(R * most + N, dtype=torch.int32, device="cuda")
    table, seq = arena[:R * most].view(R, most), arena[:R]
    _refused(sv, p, [arena], lambda: call(dict(fresh(), free_blocks=arena[R * most - 1:]), table=table))
    _refused(sv, p, [arena], lambda: call(dict(fresh(), free_blocks=arena[:N]), seq=seq))
    _refused(sv, p, [arena], lambda: call(dict(fresh(), block_table=table), seq=seq))
    for bad in (dict(free_blocks=arena[:N], block_table=table), dict(free_blocks=arena[:N], status=arena[N - 1:N + 2]),
                dict(free_blocks=arena[:N], free_count=arena[:1]), dict(block_table=table, status=arena[1:4])):
        _refused(sv, p, [*inputs, arena], lambda: call(dict(fresh(), **bad)))
    ws = torch.zeros(sv.cache_compact_workspace(N) // 4, dtype=torch.int32, device="cuda")
    _refused(sv, p, [*inputs, ws], lambda: call(dict(fresh(), status=ws[3:6]), ws=ws))
    _refused(sv, p, [ws], lambda: call(fresh(), ws=ws, seq=ws[3:6]))
    got = call(dict(block_table=table, free_blocks=arena[R * most:], free_count=torch.zeros_like(t["count"])), ws=ws)
    torch.cuda.synchronize()
    want = call(None)
    assert torch.equal(got["block_table"], want["block_table"]) and torch.equal(got["free_blocks"], want["free_blocks"])
