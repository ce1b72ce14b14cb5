"""Calls with stream=: what they allocate must not be memory that the caller's stream still uses, nor become it."""
import pytest
import torch

from tests.test_gpu_cache import Case, _commit_case, _i32

pytestmark = pytest.mark.gpu

SLEEP = 200_000_000  # cycles, a tenth of a second: far longer than what the host does meanwhile


def _blocks_of(nbytes):
    """New tensors of the current stream of this size, one of which gets a block of it that was just given back."""
    return [torch.full((nbytes,), 3, dtype=torch.uint8, device="cuda") for _ in range(8)]


def _check_workspace(call, nbytes):
    """While the call waits on its stream, its workspace is not handed to the caller's stream."""
    want = call(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SLEEP)
    got = call(s)
    others = _blocks_of(nbytes)
    s.synchronize()
    torch.cuda.synchronize()
    assert all((t == 3).all() for t in others)
    assert all(torch.equal(got[name], want[name]) for name in want)


def _check_outputs(call, between=0):
    """An output is not laid over what the caller's stream has still to read, nor over by the call's stream before the
    caller's has read it.  between: bytes of one that is not among those returned."""
    want = call(None)
    torch.cuda.synchronize()
    sizes = {t.untyped_storage().nbytes() for t in want.values()} | ({between} if between else set())
    s = torch.cuda.Stream()
    for n in sizes:
        old = _blocks_of(n)
        torch.cuda.synchronize()
        torch.cuda._sleep(SLEEP)
        copies = [t.clone() for t in old]
        del old
        got = call(s)
        torch.cuda.synchronize()
        assert all((t == 3).all() for t in copies)
    assert all(torch.equal(got[name], want[name]) for name in want)

    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(SLEEP)
    copies = {name: t.clone() for name, t in got.items()}
    del got
    with torch.cuda.stream(s):
        others = [t for n in sizes for t in _blocks_of(n)]
    torch.cuda.synchronize()
    assert all(torch.equal(copies[name], want[name]) for name in want) and all((t == 3).all() for t in others)


def _attention(sv):
    c = Case([900, 3000, 33], [9, 9, 9], 8, 2, 128, seed=13)
    kv, cu = _i32(c.kv), _i32(c.cu)

    def call(stream):
        return sv.tree_attention(c.q, c.kc, c.vc, c.table, kv, cu, 9, scale=c.scale, with_lse=True, with_status=True,
                                 stream=stream)

    return call, sv.tree_attention_workspace(3, c.T, 9, 8, 2, 128, c.table.shape[1] * 16)


def test_attention_workspace_belongs_to_the_stream(sv):
    _check_workspace(*_attention(sv))


def test_attention_outputs_belong_to_the_stream(sv):
    _check_outputs(_attention(sv)[0])


def test_table_outputs_belong_to_the_stream(sv):
    R, n = 40, 33
    seq, new, free, count = _i32([17] * R), _i32([n] * R), _i32(range(500)), _i32([500])
    table = torch.zeros((R, 8), dtype=torch.int32, device="cuda")
    parent = _i32([j - 1 for j in range(n)] * R)
    _check_outputs(lambda s: sv.step_tables(seq, new, table, free, count, 16, R * n, parent=parent, mask_words=2,
                                            stream=s))


def test_rope_outputs_belong_to_the_stream(sv):
    c = Case([40], [9], 8, 2, 64)
    k, position, slot = c.q[:, :2].contiguous(), _i32(range(9)), torch.full((9,), -1, dtype=torch.int64, device="cuda")
    freqs = sv.rope_freqs(64)
    _check_outputs(lambda s: dict(q=sv.rope_cache(c.q, k, k, position, slot, freqs, c.kc, c.vc, stream=s)))


def test_commit_outputs_belong_to_the_stream(sv):
    c = _commit_case(40, 1, 4, 1, 2, 64, 16, seed=3)
    args = [_i32(c[name]) for name in ("table", "seq", "kv", "cu", "accept")]
    free, count = _i32(c["free"]), _i32([c["count"]])
    _check_outputs(lambda s: sv.cache_commit(c["kc"][0], c["vc"][0], *args, 4, free, count, stream=s))


def test_calls_without_requests_keep_to_the_stream(sv):
    """Their fills and copies read the inputs on the given stream, not ahead of it."""
    none, table = _i32([]), torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    free, count = _i32(range(8)), _i32([0])
    caches = torch.zeros((8, 8, 1, 8), dtype=torch.bfloat16, device="cuda")
    calls = [lambda s: sv.step_tables(none, none, table, free, count, 8, 5, stream=s),
             lambda s: sv.cache_commit(caches, caches, table, none, none, _i32([0]), none, 2, free, count, stream=s)]
    for call in calls:
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            count.fill_(0)
            torch.cuda._sleep(SLEEP)
            count.fill_(7)  # ahead of the call on its stream
        got = call(s)
        torch.cuda.synchronize()
        assert got["free_count"].item() == 7


# --- verification ------------------------------------------------------------------------------------------------
R, K, V = 16, 4, 5000


def _logits(rows, width, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, width, generator=g, device="cuda") * 3


def _ids(*shape, top=V, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(top, shape, generator=g, device="cuda", dtype=torch.int32)


def _greedy(sv):
    x, draft = _logits(R * (1 + 2 * K), V, 1), _ids(R, 2, K)
    return lambda s: sv.verify_greedy(x, R, K, 2, draft, stream=s), sv.verify_greedy_workspace(R, K, 2, V)


def _greedy_top2(sv):
    x, draft = _logits(R * (1 + 2 * K), V, 2), _ids(R, 2, K)
    return lambda s: sv.verify_greedy_top2(x, R, K, 2, draft, stream=s), sv.verify_greedy_top2_workspace(R, K, 2, V)


def _sample(sv):
    x, d, draft = _logits(R * (K + 1), V, 3), _logits(R * K, V, 4), _ids(R, K)
    seeds, temp = torch.arange(R, device="cuda"), torch.full((R,), 0.8, device="cuda")
    return (lambda s: sv.verify_sample(x, d, None, R, K, draft, seeds, temp, stream=s),
            sv.verify_sample_workspace(R, K, V, V))


def _cfg(sv):
    S, W = 3, 1024
    x, y, d = _logits(R * (K + 1) * S, W, 5), _logits(R * (K + 1) * S, W, 6), _logits(R * K * S, W, 7)
    draft = _ids(R, K, S, top=W) + torch.arange(S, dtype=torch.int32, device="cuda") * W
    seeds, temp = torch.arange(R, device="cuda"), torch.full((R,), 0.8, device="cuda")

    def call(s):
        return sv.cfg_merge_sample(x, y, [0, W, 2 * W], None, S, W, 3.0, d, R, K, draft, seeds, temp, stream=s)

    return call, sv.cfg_merge_sample_workspace(R, K, S, W)


def _modality(sv):
    x = _logits(R, V, 8)
    return lambda s: sv.infer_modality(x, [0, 1000, 4000, V], stream=s), sv.load().sv_infer_modality_workspace(R, V)


def _scan(sv):
    accept, draft, fix = _ids(R, K, top=2).to(torch.uint8), _ids(R, K), _ids(R, K + 1)
    return lambda s: sv.accept_scan(accept, draft, fix, stream=s), 0


def _lookup(sv):
    pool, suffix = _ids(R, 200, top=20), _ids(R, 4, top=20)
    used = torch.full((R,), 200, dtype=torch.int32, device="cuda")
    return lambda s: sv.pool_lookup(pool, used, suffix, 8, stream=s), 0


@pytest.mark.parametrize("make", [_greedy, _greedy_top2, _sample, _cfg, _modality])
def test_verification_workspaces_belong_to_the_stream(sv, make):
    _check_workspace(*make(sv))


@pytest.mark.parametrize("make", [_greedy, _greedy_top2, _sample, _cfg, _modality, _scan, _lookup])
def test_verification_outputs_belong_to_the_stream(sv, make):
    _check_outputs(make(sv)[0])


def test_plans_belong_to_the_stream(sv):
    """A plan has bytes that nothing writes or reads, so it is compared by what comes of it."""
    Vd = 1000
    d2t = torch.randperm(V, device="cuda")[:Vd].sort().values.to(torch.int32)
    x, d, draft = _logits(R * (K + 1), V, 3), _logits(R * K, Vd, 4), d2t[_ids(R, K, top=Vd).long()]
    seeds, temp = torch.arange(R, device="cuda"), torch.full((R,), 0.8, device="cuda")

    def call(s):
        return sv.verify_sample(x, d, d2t, R, K, draft, seeds, temp, plan=sv.d2t_plan(d2t, V, stream=s), stream=s)

    _check_outputs(call, sv.d2t_plan(d2t, V).numel())
