"""The cache operators where steps are out of the ordinary: requests that take no part beside others."""
import numpy as np
import pytest
import torch

from tests.test_gpu_cache import Case, _commit_case, _i32, _np, _same, branch_parents

pytestmark = pytest.mark.gpu


# --- attention: requests without keys among others ---------------------------------------------------------------
def _without_keys(R, n, Hq, Hk, D, every, tail, longest, tree, seed):
    """Requests of n tokens, of which some were refused by the step's tables: kv_len 0, though their tokens stay."""
    rng = np.random.default_rng(seed)
    ctx = rng.integers(100, longest, R).tolist()
    kv = [0 if r % every == every - 2 or r >= R - tail else ctx[r] + n for r in range(R)]
    par = [branch_parents(1, n - 1)] * R if tree else None
    return Case(ctx, [n] * R, Hq, Hk, D, torch.bfloat16, 16, parents=par, seed=seed, kv=kv), kv


# Sizes that give several items to a CTA, so that items without keys follow ones with keys in one CTA's share: with one
# row tile, with several (masked and as chains), and with two accumulators of each stream (heads of 64) or one.
@pytest.mark.parametrize("R,n,Hq,Hk,D,every,tail,longest,tree", [
    (64, 9, 32, 8, 128, 9, 1, 8000, False), (48, 9, 16, 8, 64, 4, 3, 900, True), (200, 1, 8, 4, 64, 5, 2, 140, False),
    (48, 70, 32, 8, 128, 4, 3, 900, True), (48, 70, 32, 8, 64, 4, 3, 900, False), (40, 300, 8, 4, 128, 4, 2, 400, True)])
def test_attention_requests_without_keys_among_others(sv, R, n, Hq, Hk, D, every, tail, longest, tree):
    c, kv = _without_keys(R, n, Hq, Hk, D, every, tail, longest, tree, seed=R + n)
    out = dict(out=torch.full_like(c.q, 7.0), lse=torch.full((c.T, Hq), 7.0, device="cuda"),
               status=torch.full((R,), -1, dtype=torch.int32, device="cuda"))
    got = c.run(sv, out=out)
    assert (got["status"] == 0).all()
    none = torch.tensor([x == 0 for x in kv]).repeat_interleave(n).cuda()
    assert (got["out"][none] == 0).all() and torch.isneginf(got["lse"][none]).all()
    # the others have the bits that they have without them
    rest = [r for r in range(R) if kv[r] > 0]
    rows = torch.cat([torch.arange(r * n, r * n + n) for r in rest]).cuda()
    alone = sv.tree_attention(c.q[rows], c.kc, c.vc, c.table[rest].contiguous(), _i32([kv[r] for r in rest]),
                              _i32(np.arange(len(rest) + 1) * n), n,
                              mask=None if c.mask is None else _i32(c.mask)[rows].contiguous(), scale=c.scale,
                              with_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(got["out"][rows], alone["out"]) and torch.equal(got["lse"][rows], alone["lse"])
    c.check(got, sorted(rest, key=lambda r: kv[r])[:2])


@pytest.mark.parametrize("n,D", [(5, 128), (90, 64)])
def test_attention_where_only_few_requests_have_keys(sv, n, D):
    """Long rows of items without keys, and a batch that has nothing else."""
    R = 600 if n == 5 else 60
    for keep in ([], [0], [R // 2], [0, R // 3, R - 1]):
        kv = [200 + n if r in keep else 0 for r in range(R)]
        c = Case([200] * R, [n] * R, 8, 4, D, torch.float16, 16, seed=n, kv=kv)
        out = dict(out=torch.full_like(c.q, 7.0), lse=torch.full((c.T, 8), 7.0, device="cuda"),
                   status=torch.full((R,), -1, dtype=torch.int32, device="cuda"))
        got = c.run(sv, out=out)
        assert (got["status"] == 0).all()
        none = torch.tensor([x == 0 for x in kv]).repeat_interleave(n).cuda()
        assert (got["out"][none] == 0).all() and torch.isneginf(got["lse"][none]).all()
        c.check(got, keep)


# --- attention: a wait that gave up -------------------------------------------------------------------------------
@pytest.mark.parametrize("new,D,dtype", [([9, 9, 1, 4], 128, torch.bfloat16), ([70, 1, 300, 9], 128, torch.float16),
                                         ([33, 33, 2, 1], 64, torch.bfloat16), ([300, 65, 9, 140], 64, torch.bfloat16)])
def test_attention_that_gave_up_says_so(sv, new, D, dtype):
    """One CTA gives up at its first wait: every request is reported, no row looks like a result, the next call is
    right."""
    c = Case([3000, 40, 900, 0], new, 16, 4, D, dtype, 16, seed=D + sum(new))
    want = c.run(sv, with_status=True)
    assert (want["status"] == 0).all()
    kv, cu = _i32(c.kv), _i32(c.cu)
    nbytes = sv.tree_attention_workspace(c.R, c.T, c.max_tokens, 16, 4, D, c.table.shape[1] * 16)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    for cta in (0, 75, torch.cuda.get_device_properties(0).multi_processor_count - 1):
        out, lse = torch.zeros_like(c.q), torch.zeros(c.T, 16, device="cuda")
        status = torch.zeros(c.R, dtype=torch.int32, device="cuda")
        rc = sv.load().sv_selftest_tree_attention_stop(
            sv.heads_of(c.q), sv.cache_of(c.kc, c.vc), c.table.data_ptr(), c.table.shape[1], kv.data_ptr(),
            cu.data_ptr(), c.R, c.max_tokens, None, 0, c.scale, sv.heads_of(out), lse.data_ptr(), status.data_ptr(),
            ws.data_ptr(), nbytes, cta, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert rc == 0 and (status == sv.ST_TIMEOUT).all()
        assert torch.isnan(out.float()).all() and torch.isnan(lse).all()
        again = c.run(sv, workspace=ws, with_status=True)
        assert (again["status"] == 0).all()
        assert torch.equal(again["out"], want["out"]) and torch.equal(again["lse"], want["lse"])


@pytest.mark.parametrize("new,D", [([9, 9, 1, 4], 128), ([70, 1, 300, 9], 128), ([300, 65, 9, 140], 64),
                                   ([1, 1, 1, 1], 64)])
def test_attention_that_gave_up_ends_at_once(sv, new, D):
    """What a CTA waits for before it leaves is what is in flight: the call takes nowhere near a wait's limit, 2 s."""
    c = Case([3000, 40, 900, 0], new, 16, 4, D, torch.bfloat16, 16, seed=D + sum(new))
    kv, cu = _i32(c.kv), _i32(c.cu)
    nbytes = sv.tree_attention_workspace(c.R, c.T, c.max_tokens, 16, 4, D, c.table.shape[1] * 16)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(c.q)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for cta in range(0, 152, 19):
        start.record()
        rc = sv.load().sv_selftest_tree_attention_stop(
            sv.heads_of(c.q), sv.cache_of(c.kc, c.vc), c.table.data_ptr(), c.table.shape[1], kv.data_ptr(),
            cu.data_ptr(), c.R, c.max_tokens, None, 0, c.scale, sv.heads_of(out), None, None, ws.data_ptr(), nbytes, cta,
            torch.cuda.current_stream().cuda_stream)
        end.record()
        torch.cuda.synchronize()
        assert rc == 0 and start.elapsed_time(end) < 500, cta


# --- commit: blocks outside the pool ------------------------------------------------------------------------------
def _commit_plain(c, k, path):
    """What is kept, one token and one block at a time: a block outside the pool holds nothing and is not given back."""
    kc, vc, free = _np(c["kc"]).copy(), _np(c["vc"]).copy(), c["free"].copy()
    nb, bs, top = kc.shape[1], kc.shape[2], c["count"]
    seq, status = np.array(c["seq"], np.int32), np.zeros(len(c["seq"]), np.int32)
    for r in range(len(seq)):
        L, kv, table = int(c["seq"][r]), int(c["kv"][r]), c["table"][r]
        n = int(c["cu"][r + 1] - c["cu"][r])
        if n <= 0 or L + n != kv:
            continue
        a = min(max(int(c["accept"][r]), 0), k)
        if any(not 0 <= table[(L + j) // bs] < nb for j in range(n)):
            status[r] = 2048
        for cache in (kc, vc):
            for i in range(a):
                src, dst = L + int(path[r, i]), L + 1 + i
                if 0 <= table[src // bs] < nb and 0 <= table[dst // bs] < nb:
                    cache[:, table[dst // bs], dst % bs] = cache[:, table[src // bs], src % bs]
        seq[r] = L + 1 + a
        for b in range(-(-int(seq[r]) // bs), -(-kv // bs)):
            if 0 <= table[b] < nb:
                free[top] = table[b]
                top += 1
    return dict(k=kc, v=vc, seq_len=seq, free=free, free_count=np.array([top], np.int32), status=status)


@pytest.mark.parametrize("R,bs", [(12, 8), (300, 8), (40, 16)])
@pytest.mark.parametrize("by_path", [False, True])
def test_commit_gives_no_block_back_that_is_outside_the_pool(sv, R, bs, by_path):
    """Two branches of 20 drafts; entries of many tables replaced among the committed, kept and surplus blocks."""
    k, n = 20, 41
    c = _commit_case(R, 2, k, 2, 2, 16, bs, seed=R)
    rng = np.random.default_rng(R + 1)
    nb = c["kc"].shape[1]
    for r in range(0, R, 2):
        held = -(-int(c["kv"][r]) // bs)
        for b in rng.choice(held, min(held, 3), replace=False) if held else []:
            c["table"][r, b] = rng.choice([-1, -(1 << 31), nb, nb + 7, (1 << 31) - 1])
    if by_path:
        path = np.stack([np.sort(rng.choice(np.arange(1, n), k, replace=False)) for _ in range(R)]).astype(np.int32)
    else:
        path = 1 + c["branch"][:, None] * k + np.arange(k)
    want = _commit_plain(c, k, path)
    assert (want["status"] == 2048).any() and (want["status"] == 0).any()
    free = _i32(c["free"])
    got = sv.cache_commit(c["kc"], c["vc"], _i32(c["table"]), _i32(c["seq"]), _i32(c["kv"]), _i32(c["cu"]),
                          _i32(c["accept"]), k, free, _i32([c["count"]]),
                          branch=None if by_path else _i32(c["branch"]), path=_i32(path) if by_path else None)
    torch.cuda.synchronize()
    for name in ("seq_len", "free_count", "status"):
        _same(got[name], want[name], name)
    _same(free, want["free"], "free")
    np.testing.assert_array_equal(_np(c["kc"]), want["k"])
    np.testing.assert_array_equal(_np(c["vc"]), want["v"])


def test_a_block_outside_the_pool_reaches_no_other_request(sv):
    """A request with a bad entry is committed; the next step's tokens of another request have slots all the same."""
    bs, nb, k = 8, 6, 15
    table = _i32([[0, -1, -1, -1], [1, -1, -1, -1]])
    seq, free, count = _i32([8, 8]), _i32([2, 3, 4, 5, -1, -1]), _i32([4])
    kc, vc = (torch.zeros(nb, bs, 1, 8, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    step = sv.step_tables(seq, _i32([1 + k, 0]), table, free, count, bs, 1 + k)
    assert table[0].tolist() == [0, 5, 4, -1] and step["free_count"].item() == 2
    table[0, 2] = nb + 3
    kept = sv.cache_commit(kc, vc, table, seq, step["kv_len"], step["cu_tokens"], _i32([0, 0]), k, free,
                           step["free_count"])
    assert kept["status"].tolist() == [2048, 0] and kept["free_count"].item() == 2
    step = sv.step_tables(kept["seq_len"], _i32([0, 9]), table, free, kept["free_count"], bs, 9)
    assert step["status"].tolist() == [0, 0] and (step["slot"] >= 0).all()
