"""The cache operators where steps are out of the ordinary: requests that take no part beside others."""
import numpy as np
import pytest
import torch

from tests.test_gpu_cache import Case, _i32, branch_parents

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
    c.check(got, [rest[0], rest[-1]])


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
