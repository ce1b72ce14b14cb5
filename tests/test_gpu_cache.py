"""The cache operators on the GPU against the plain 64-bit forms: tables and commits exactly, rotations and
attention within bounds that follow from the arithmetic (no measured slack)."""
import numpy as np
import pytest
import torch

from tests import cache_plain as plain

pytestmark = pytest.mark.gpu

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a unit in the last place, relative
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}        # the same below fp16's normal range, absolute


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


def _same(got, want, name):
    np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=name)


def branch_parents(branches, k):
    par = [-1]
    for b in range(branches):
        par += [0 if j == 0 else b * k + j for j in range(k)]
    return par


# --- step tables -----------------------------------------------------------------------------------------------
def _check_tables(sv, seq, new, bs, mb, nb, count, T, parent=None, words=0, spoil=None, seed=0):
    rng = np.random.default_rng(seed)
    R = len(seq)
    table = np.full((R, mb), -7, np.int32)
    order = rng.permutation(nb).astype(np.int32)
    used = 0
    for r in range(R):
        held = -(-max(int(seq[r]), 0) // bs)
        for i in range(min(held, mb)):
            table[r, i] = order[used % nb]
            used += 1
    free = rng.permutation(nb).astype(np.int32)
    if spoil is not None:
        table[spoil] = nb + 3
    want = plain.tables(seq, new, table, free, count, bs, T, nb, parent, words)
    dt = _i32(table)
    got = sv.step_tables(_i32(seq), _i32(new), dt, _i32(free), _i32([count]), bs, T,
                         parent=None if parent is None else _i32(parent), mask_words=words)
    again = sv.step_tables(_i32(seq), _i32(new), dt, _i32(free), _i32([count]), bs, T,
                           parent=None if parent is None else _i32(parent), mask_words=words)
    torch.cuda.synchronize()
    for g in (got, again):
        for name in ("status", "cu_tokens", "kv_len", "slot", "position", "free_count"):
            _same(g[name], want[name], name)
        if parent is not None:
            _same(g["mask"], want["mask"], "mask")
    _same(dt, want["block_table"], "block_table")
    return want


@pytest.mark.parametrize("bs", [1, 8, 16, 24, 128])
@pytest.mark.parametrize("R", [1, 2, 37, 700])
def test_tables_chain(sv, R, bs):
    rng = np.random.default_rng(R * 1000 + bs)
    seq = rng.integers(0, 300, R)
    new = rng.integers(0, 12, R)
    seq[0] = 0
    if R > 2:
        new[1], seq[2] = 0, bs  # a request that sits out; a full last block
    mb = -(-320 // bs)
    need = int((-(-(seq + new) // bs) + seq // -bs).sum())
    _check_tables(sv, seq, new, bs, mb, need + 50, need, int(new.sum()) + 5, seed=R)


@pytest.mark.parametrize("branches,k", [(1, 0), (1, 8), (2, 32), (8, 4), (3, 31), (8, 256), (1, 31), (1, 32)])
def test_tables_branch_trees(sv, branches, k):
    R, n = 5, 1 + branches * k
    par = np.tile(branch_parents(branches, k), R)
    seq = np.array([0, 1, 15, 16, 1000])
    _check_tables(sv, seq, np.full(R, n), 16, 260, 2000, 1500, R * n, par, -(-n // 32) + 1)


def test_tables_random_trees_and_bad_parents(sv):
    rng = np.random.default_rng(3)
    new = np.array([1, 7, 40, 0, 33, 64, 65])
    par = np.concatenate([[rng.integers(-1, j) if j else -1 for j in range(n)] for n in new]).astype(np.int64)
    seq = np.array([0, 3, 200, 9, 15, 16, 17])
    want = _check_tables(sv, seq, new, 8, 40, 200, 150, int(new.sum()), par, 3)
    assert not want["status"].any()
    par[3], par[20], par[70] = 5, 400, -9  # not below the token, not one of the request's, no parent at all
    want = _check_tables(sv, seq, new, 8, 40, 200, 150, int(new.sum()), par, 3)
    assert (want["status"] == 512).sum() == 3


def test_tables_that_run_out(sv):
    seq, new = np.full(40, 30), np.full(40, 9)  # every request needs one block of 16... from the third token on
    for count in (0, 1, 17, 39, 40, 64):
        want = _check_tables(sv, seq, new, 16, 3, 64, count, 400)
        assert (want["status"] == 256).sum() == max(0, 40 - count)
    # the packed arrays are too short: from there on nobody takes part, but those without tokens do
    new = np.where(np.arange(40) % 3 == 0, 0, 9)
    want = _check_tables(sv, seq, new, 16, 3, 64, 64, 100)
    assert (want["status"] == 256).any() and want["free_count"][0] == 64 - 11


def test_tables_bad_lengths_and_blocks(sv):
    seq = np.array([5, -1, 5, 100, 40, 2])
    new = np.array([3, 4, -2, 90, 3, 3])
    want = _check_tables(sv, seq, new, 8, 20, 100, 50, 200)
    assert want["status"].tolist() == [0, 1024, 1024, 1024, 0, 0]
    want = _check_tables(sv, seq, new, 8, 20, 100, 50, 200, spoil=(0, 0))
    assert want["status"][0] == 2048
    # a tree wider than its mask
    par = np.tile(branch_parents(1, 39), 2)
    want = _check_tables(sv, [4, 4], [40, 40], 8, 20, 100, 50, 80, par, 1)
    assert want["status"].tolist() == [1024, 1024]


# --- rotary positions and cache writes ----------------------------------------------------------------------------
def _rope_case(T, Hq, Hk, D, dtype, bs=16, seed=0, fused=True, head_major=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if fused:
        x = torch.randn(T, Hq + 2 * Hk, D, generator=g, device="cuda").to(dtype)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    else:
        q, k, v = (torch.randn(T, h, D, generator=g, device="cuda").to(dtype) for h in (Hq, Hk, Hk))
    nb = -(-T // bs) + 3
    shape = (nb, Hk, bs, D) if head_major else (nb, bs, Hk, D)
    kc = torch.full(shape, 7.0, dtype=dtype, device="cuda")
    vc = torch.full(shape, 7.0, dtype=dtype, device="cuda")
    if head_major:
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    slot = torch.randperm(nb * bs, generator=g, device="cuda")[:T]
    return q, k, v, kc, vc, slot


def _rope_bound(x, half, mscale, dtype, interleaved):
    """|error| <= rounding to dtype, and for x and y of a pair (|x| + |y|) m e: e = 2^-24 half turns pi of the angle's
    last bit and its conversion, two units of the sine, two of the products."""
    D = x.shape[-1]
    first = np.arange(half) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    pair = np.zeros_like(x)
    if half:
        tot = np.abs(x[..., first]) + np.abs(x[..., second])
        pair[..., first] = pair[..., second] = tot
    assert pair.shape[-1] == D
    return abs(mscale) * pair * (np.pi * 2.0 ** -24 + 4 * 2.0 ** -23)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [
    (1, 1, 1, 8, 8), (1, 32, 8, 128, 128), (9, 28, 4, 128, 64), (65, 6, 3, 96, 96), (33, 5, 5, 80, 20),
    (17, 4, 2, 64, 0), (40, 8, 1, 72, 36), (300, 3, 3, 16, 2), (5, 64, 2, 128, 48), (7, 2, 1, 24, 24)])
def test_rope(sv, T, Hq, Hk, D, rot, interleaved, dtype):
    q, k, v, kc, vc, slot = _rope_case(T, Hq, Hk, D, dtype, seed=T + D, fused=T != 65, head_major=T == 33)
    rng = np.random.default_rng(T)
    pos = rng.integers(0, 131072, T).astype(np.int32)
    pos[0] = 0
    if T > 4:
        slot[2], slot[3] = -1, kc.shape[0] * kc.shape[1]  # neither is written
    freqs = sv.rope_freqs(rot, 10000.0)
    mscale = 1.0 if T != 9 else 1.2772588722239782
    before = kc.clone()
    got = sv.rope_cache(q, k, v, _i32(pos), slot, freqs, kc, vc, interleaved=interleaved, mscale=mscale)
    torch.cuda.synchronize()
    ang = plain.turns(freqs.cpu().tolist(), pos)
    u = UNIT[dtype]
    flat_k = kc.reshape(-1, Hk, D)
    flat_v = vc.reshape(-1, Hk, D)
    live = ((slot >= 0) & (slot < flat_k.shape[0])).cpu().numpy()
    for name, x, y in (("q", q, got), ("k", k, flat_k[slot.clamp(0, flat_k.shape[0] - 1)])):
        want = plain.rotate(_np(x), ang, interleaved, mscale)
        tol = _rope_bound(_np(x), rot // 2, mscale, dtype, interleaved)
        tol = tol + u * (np.abs(want) + tol) + TINY[dtype]
        err = np.abs(_np(y) - want)
        rows = live if name == "k" else slice(None)
        assert (err[rows] <= tol[rows]).all(), (name, (err / tol)[rows].max())
        if 2 * (rot // 2) < D:  # what is not rotated passes as it is
            assert torch.equal(y[rows if name == "q" else torch.from_numpy(live).cuda()][..., rot:],
                               x[rows if name == "q" else torch.from_numpy(live).cuda()][..., rot:])
    lv = torch.from_numpy(live).cuda()
    assert torch.equal(flat_v[slot[lv]], v[lv])
    untouched = torch.ones(flat_k.shape[0], dtype=torch.bool, device="cuda")
    untouched[slot[lv]] = False
    assert torch.equal(flat_k[untouched], before.reshape(-1, Hk, D)[untouched])
    # in place
    q2 = q.clone() if q.is_contiguous() else q
    same = sv.rope_cache(q2, k, v, _i32(pos), slot, freqs, kc, vc, interleaved=interleaved, mscale=mscale, q_out=q2)
    torch.cuda.synchronize()
    assert torch.equal(same, got)


def test_rope_keeps_its_angle_at_long_positions(sv):
    """Relative positions decide: q at p + d and k at p give the same product for every p (up to rounding)."""
    D = 128
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, 1, D, generator=g, device="cuda").to(torch.float16).expand(2, 1, D).contiguous()
    freqs = sv.rope_freqs(D, 500000.0)
    dots = []
    for p in (0, 1000, 131072, 10_000_000, 2_000_000_000):
        kc = torch.zeros(1, 8, 1, D, dtype=torch.float16, device="cuda")
        q = sv.rope_cache(x, x, x, _i32([p + 37, p]), torch.tensor([0, 1], device="cuda"), freqs, kc, kc.clone())
        torch.cuda.synchronize()
        dots.append(float((_np(q)[0, 0] * _np(kc)[0, 1, 0]).sum()))
    size = float((_np(x)[0, 0] ** 2).sum())
    # both factors carry a rounding of 2^-11 and an angle error below 2^-21
    assert max(dots) - min(dots) <= 2 * (2 * 2.0 ** -11 + 2.0 ** -20) * size


# --- attention -------------------------------------------------------------------------------------------------
class Case:
    """Requests with caches of their own blocks; every slot that holds no key of theirs is NaN."""

    def __init__(self, ctx, new, Hq, Hk, D, dtype=torch.bfloat16, bs=16, parents=None, seed=0, head_major=False,
                 sharp=1.0, words=None, spare=0, stale=float("nan"), kv=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ctx, self.new, self.Hq, self.Hk, self.D, self.dtype, self.bs = list(ctx), list(new), Hq, Hk, D, dtype, bs
        R = self.R = len(ctx)
        kv = self.kv = [c + n for c, n in zip(ctx, new)] if kv is None else list(kv)
        mb = max(1, max(-(-x // bs) for x in kv)) + spare
        nb = sum(-(-x // bs) for x in kv) + 2
        order = rng.permutation(nb)
        table = np.full((R, mb), nb + 5, np.int32)
        shape = (nb, Hk, bs, D) if head_major else (nb, bs, Hk, D)
        self.kc = torch.full(shape, stale, dtype=dtype, device="cuda")
        self.vc = torch.full(shape, stale, dtype=dtype, device="cuda")
        if head_major:
            self.kc, self.vc = self.kc.permute(0, 2, 1, 3), self.vc.permute(0, 2, 1, 3)
        self.K, self.V, at = [], [], 0
        for r in range(R):
            n = -(-kv[r] // bs)
            table[r, :n] = order[at:at + n]
            ids = torch.from_numpy(order[at:at + n].copy()).cuda()
            at += n
            for cache, keep in ((self.kc, self.K), (self.vc, self.V)):
                x = torch.randn(kv[r], Hk, D, generator=g, device="cuda").to(dtype)
                keep.append(x)
                if n:
                    pos = torch.arange(kv[r], device="cuda")
                    cache[ids[pos // bs], pos % bs] = x
        self.table = _i32(table)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = self.T = int(self.cu[-1])
        self.q = (torch.randn(T, Hq, D, generator=g, device="cuda") * sharp).to(dtype)
        self.max_tokens = max(new) if new else 0
        self.mask = None
        if parents is not None:
            words = words if words is not None else max(1, -(-self.max_tokens // 32))
            m = np.zeros((T, words), np.uint32)
            for r in range(R):
                for j in range(new[r]):
                    t = self.cu[r] + j
                    p = parents[r][j]
                    if p >= 0:
                        m[t] = m[self.cu[r] + p]
                    if j < 32 * words:
                        m[t, j // 32] |= np.uint32(1 << (j % 32))
            self.mask = m.view(np.int32)
        self.scale = D ** -0.5

    def run(self, sv, **more):
        got = sv.tree_attention(self.q, self.kc, self.vc, self.table, _i32(self.kv), _i32(self.cu), self.max_tokens,
                                mask=None if self.mask is None else _i32(self.mask), scale=self.scale, with_lse=True,
                                **more)
        torch.cuda.synchronize()
        return got

    def want(self, r):
        t0, t1 = self.cu[r], self.cu[r + 1]
        return plain.attention(_np(self.q)[t0:t1], _np(self.K[r]), _np(self.V[r]), self.kv[r] - self.new[r],
                               self.new[r], self.scale, None if self.mask is None else self.mask[t0:t1])

    def check(self, got, requests=None):
        u = UNIT[self.dtype]
        for r in range(self.R) if requests is None else requests:
            if self.new[r] == 0:
                continue
            out, lse, spread, reach = self.want(r)
            t0, t1 = self.cu[r], self.cu[r + 1]
            # a score is off by at most (D + 2) 2^-24 of its products' absolute sum, a probability relatively by that,
            # the exponential and the sums; it is rounded once to the cache's type and the result once to q's
            ds = (self.D + 2) * 2.0 ** -24 * reach
            rel = 2 * ds + (self.kv[r] + 64) * 2.0 ** -24
            tol = spread * (u + rel[..., None]) * (1 + 2 * u) + u * np.abs(out) + \
                TINY[self.dtype] * (1 + self.kv[r] * float(self.V[r].abs().nan_to_num(0, 0, 0).max()))
            err = np.abs(_np(got["out"])[t0:t1] - out)
            assert (err <= tol).all(), (r, (err / np.maximum(tol, 1e-300)).max())
            gl = _np(got["lse"])[t0:t1]
            np.testing.assert_array_equal(np.isneginf(gl), np.isneginf(lse))
            ok = ~np.isneginf(lse)
            # ln 2 times a base-2 result rounds at the result's own size
            err = np.abs(gl - np.where(ok, lse, 0))[ok]
            assert (err <= (rel + 2.0 ** -22 * (1 + np.abs(np.where(ok, lse, 0)) + reach))[ok]).all(), r


LENGTHS = [0, 1, 7, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 500, 1025]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bs", [8, 16, 24, 48, 64, 128, 256])
def test_attention_single_tokens_at_every_edge(sv, bs, dtype):
    c = Case(LENGTHS, [1] * len(LENGTHS), 8, 2, 64, dtype, bs, seed=bs)
    c.check(c.run(sv))


@pytest.mark.parametrize("D", [8, 24, 64, 72, 96, 128])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (7, 1), (6, 3), (28, 4), (40, 2)])
def test_attention_heads(sv, Hq, Hk, D):
    c = Case([0, 130, 300], [3, 9, 1], Hq, Hk, D, torch.bfloat16 if D != 72 else torch.float16, 16, seed=D + Hq)
    c.check(c.run(sv))


@pytest.mark.parametrize("branches,k", [(1, 8), (2, 32), (8, 4), (3, 43), (8, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_trees(sv, branches, k, dtype):
    n = 1 + branches * k
    par = branch_parents(branches, k)
    ctx = [0, 1, 100, 127, 250, 511]
    c = Case(ctx, [n] * len(ctx), 8, 2, 128, dtype, 32, parents=[par] * len(ctx), seed=n)
    c.check(c.run(sv))


def test_attention_ragged_batch(sv):
    rng = np.random.default_rng(5)
    new = [0, 1, 40, 0, 33, 128, 129, 2, 300, 0]
    ctx = [10, 0, 77, 0, 1000, 5, 640, 129, 0, 3]
    par = [[int(rng.integers(-1, j)) if j else -1 for j in range(n)] for n in new]
    c = Case(ctx, new, 12, 4, 96, torch.bfloat16, 24, parents=par, seed=2)
    c.check(c.run(sv))
    c = Case(ctx, new, 12, 4, 96, torch.bfloat16, 24, seed=3)  # chains: long ones are whole prompts
    c.check(c.run(sv))


def test_attention_rows_that_see_nothing(sv):
    c = Case([0, 0, 50], [5, 3, 4], 4, 2, 64, parents=[[-1] * 5, [-1] * 3, [-1] * 4], seed=1)
    m = c.mask.copy()
    m[0] = 0            # no position before it, no bit
    m[6] = 0
    m[9] = 0            # sees the 50 committed ones
    c.mask = m
    got = c.run(sv)
    c.check(got)
    assert torch.isneginf(got["lse"][0]).all() and (got["out"][0] == 0).all()
    assert torch.isfinite(got["lse"][9]).all()


def test_attention_request_without_keys(sv):
    """kv_len 0 (a request that took no part in the step's tables), and fewer keys than tokens."""
    c = Case([0, 20], [4, 4], 4, 2, 64, seed=4, kv=[0, 24])
    got = c.run(sv)
    assert (got["out"][:4] == 0).all() and torch.isneginf(got["lse"][:4]).all()
    c.check(got, [1])
    c = Case([0, 0], [5, 9], 4, 2, 64, seed=5, kv=[3, 1])
    c.check(c.run(sv))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_hidden_keys_have_no_influence(sv, bad):
    """Drafted keys and values that only their own branch sees: the other branch's rows stay as they are."""
    par = branch_parents(2, 20)
    base = Case([70, 0], [41, 41], 8, 2, 64, parents=[par, par], seed=6)
    clean = base.run(sv)
    for what in ("k", "v"):
        c = Case([70, 0], [41, 41], 8, 2, 64, parents=[par, par], seed=6)
        cache = c.kc if what == "k" else c.vc
        for r, j in ((0, 25), (1, 30), (1, 40)):
            at = c.kv[r] - 41 + j
            cache[int(c.table[r, at // c.bs]), at % c.bs, 1, 3:] = bad
        got = c.run(sv)
        for r, j in ((0, 25), (1, 30)):
            t0 = int(c.cu[r])
            hidden = [t0 + x for x in range(41) if x < j or (x <= 20)]
            hidden = [t for t in hidden if not (t - t0 > 20 and t - t0 >= j)]
            assert torch.equal(got["out"][hidden], clean["out"][hidden]), (what, r)
            assert torch.equal(got["lse"][hidden], clean["lse"][hidden]), (what, r)
            # heads of the other key head are clean everywhere
            assert torch.equal(got["out"][t0:t0 + 41, :4], clean["out"][t0:t0 + 41, :4])
            sees = list(range(t0 + j, t0 + 41))
            if what == "v":
                x = got["out"][sees][:, 4:, 3:].float()
                assert not torch.isfinite(x).any()
                assert torch.isfinite(got["out"][sees][:, 4:, :3].float()).all()
                assert torch.equal(got["lse"][sees], clean["lse"][sees])
    assert torch.isfinite(clean["out"].float()).all()


def test_attention_sharp_and_growing_scores(sv):
    """Scores of hundreds, growing along the keys, so the running maximum moves in every part."""
    c = Case([600, 1200], [5, 3], 4, 2, 64, torch.bfloat16, 16, seed=7, sharp=4.0)
    for r in range(2):
        ramp = torch.linspace(0.1, 20.0, c.kv[r], device="cuda").view(-1, 1, 1)
        x = (c.K[r].float().abs() * ramp).to(c.dtype)
        c.K[r] = x
        pos = torch.arange(c.kv[r], device="cuda")
        c.kc[c.table[r].long()[pos // c.bs], pos % c.bs] = x
    c.q = c.q.abs()
    c.check(c.run(sv))


def test_attention_strides(sv):
    c = Case([100, 37, 260], [9, 1, 17], 8, 4, 64, torch.float16, 16, seed=8, head_major=True, spare=3)
    want = c.run(sv)
    c.check(want)
    wide = torch.randn(c.T, 3 * 8 + 4, 64, device="cuda").to(c.dtype)
    wide[:, 4:12] = c.q
    c.q = wide[:, 4:12]
    turned = torch.empty(8, c.T, 64, dtype=c.dtype, device="cuda").permute(1, 0, 2)  # heads outermost
    out = dict(out=turned, lse=torch.empty(c.T, 8, device="cuda"))
    got = c.run(sv, out=out)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


@pytest.mark.parametrize("ctx,n,Hq,Hk,D", [(5000, 9, 8, 2, 128), (20011, 1, 4, 1, 64), (40000, 65, 7, 1, 128),
                                           (9000, 1, 16, 16, 128), (70000, 2, 2, 1, 128), (3000, 257, 8, 2, 64)])
def test_attention_long(sv, ctx, n, Hq, Hk, D):
    c = Case([ctx], [n], Hq, Hk, D, torch.bfloat16, 16, seed=n)
    c.check(c.run(sv))


def test_attention_does_not_depend_on_the_batch(sv):
    """A request alone, in a batch, and in the batch reversed: the same bits (contexts long enough to be split)."""
    par = branch_parents(2, 7)
    ctx = [3000, 0, 17, 9000, 128, 640, 5000, 2000] * 3
    c = Case(ctx, [15] * len(ctx), 8, 2, 128, torch.bfloat16, 16, parents=[par] * len(ctx), seed=9)
    got = c.run(sv)
    again = c.run(sv)
    assert torch.equal(got["out"], again["out"])

    def only(rs):
        rows = torch.cat([torch.arange(15 * r, 15 * r + 15) for r in rs]).cuda()
        x = sv.tree_attention(c.q[rows], c.kc, c.vc, c.table[rs].contiguous(), _i32([c.kv[r] for r in rs]),
                              _i32(np.arange(len(rs) + 1) * 15), 15, mask=_i32(c.mask)[rows].contiguous(),
                              scale=c.scale, with_lse=True)
        torch.cuda.synchronize()
        return rows, x

    for rs in ([0], [3], [7], [4], list(range(len(ctx)))[::-1], [3, 0]):
        rows, x = only(rs)
        assert torch.equal(x["out"], got["out"][rows]) and torch.equal(x["lse"], got["lse"][rows]), rs


@pytest.mark.parametrize("D,Hq,Hk", [(128, 8, 2), (64, 28, 4), (72, 6, 6)])
def test_attention_does_not_depend_on_the_other_requests_rows(sv, D, Hq, Hk):
    """Next to a request of several row tiles, or with room for one, a request has the bits that it has alone."""
    rng = np.random.default_rng(D)
    new = [9, 300, 1, 5, 0, 129]
    ctx = [4000, 1500, 700, 128, 10, 0]
    par = [[int(rng.integers(-1, j)) if j else -1 for j in range(n)] for n in new]
    c = Case(ctx, new, Hq, Hk, D, torch.bfloat16, 16, parents=par, seed=D)
    got = c.run(sv)
    c.check(got)
    words = c.mask.shape[1]
    for r in (0, 2, 3, 5, 1):
        t0, t1 = int(c.cu[r]), int(c.cu[r + 1])
        for most in (new[r], 300):
            x = sv.tree_attention(c.q[t0:t1], c.kc, c.vc, c.table[r:r + 1], _i32([c.kv[r]]), _i32([0, new[r]]), most,
                                  mask=_i32(c.mask[t0:t1]).view(-1, words), scale=c.scale, with_lse=True)
            torch.cuda.synchronize()
            assert torch.equal(x["out"], got["out"][t0:t1]) and torch.equal(x["lse"], got["lse"][t0:t1]), (r, most)


@pytest.mark.parametrize("R", [385, 1500])
def test_attention_many_short_requests(sv, R):
    rng = np.random.default_rng(R)
    new = rng.integers(0, 4, R)
    ctx = rng.integers(0, 40, R)
    c = Case(ctx.tolist(), new.tolist(), 4, 2, 64, torch.bfloat16, 16, seed=R)
    c.check(c.run(sv))


@pytest.mark.parametrize("scale", [0.0, -0.125, 3.0])
def test_attention_scales(sv, scale):
    c = Case([300, 5, 1000], [9, 3, 70], 8, 2, 64, torch.float16, 16, seed=31)
    c.scale = scale
    c.check(c.run(sv))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_scores_that_are_not_finite(sv, bad):
    """A visible key whose score is NaN or +inf makes the whole row and its lse NaN; the rows before it stay."""
    for ctx, n, at in ((0, 1, 0), (0, 9, 4), (300, 9, 304), (2000, 9, 2004)):
        clean = Case([ctx, 40], [n, n], 4, 2, 64, seed=33)
        clean.q = clean.q.abs() + 0.5  # with a key of +inf the score is +inf
        want = clean.run(sv)
        c = Case([ctx, 40], [n, n], 4, 2, 64, seed=33)
        c.q = clean.q
        c.kc[int(c.table[0, at // c.bs]), at % c.bs, 1, 5] = bad
        got = c.run(sv)
        j = max(0, at - ctx)  # from this token on
        assert torch.isnan(got["out"][j:n, 2:].float()).all() and torch.isnan(got["lse"][j:n, 2:]).all(), (ctx, n)
        for name in ("out", "lse"):
            assert torch.equal(got[name][:j], want[name][:j]) and torch.equal(got[name][n:], want[name][n:])
            assert torch.equal(got[name][:n, :2], want[name][:n, :2])


def test_attention_bounds_of_tokens_and_masks(sv):
    """Tokens beyond max_tokens are left alone; bits beyond the mask's words count as 0."""
    par = branch_parents(1, 49)
    c = Case([30, 64], [50, 50], 4, 2, 64, parents=[par, par], seed=10, words=1)
    c.mask = np.full((100, 1), -1, np.int32)  # every token sees tokens 0..31
    c.check(c.run(sv))
    c.max_tokens = 20
    out = dict(out=torch.full_like(c.q, 5.0), lse=torch.full((100, 4), 5.0, device="cuda"))
    got = c.run(sv, out=out)
    for r in range(2):
        assert (got["out"][50 * r + 20:50 * r + 50] == 5).all() and (got["lse"][50 * r + 20:50 * r + 50] == 5).all()
    c.max_tokens = 50
    full = c.run(sv)
    keep = torch.cat([torch.arange(20), torch.arange(50, 70)]).cuda()
    assert torch.equal(got["out"][keep], full["out"][keep])


def test_attention_blocks_outside_the_pool_read_as_zeros(sv):
    c = Case([40], [2], 4, 2, 64, torch.bfloat16, 16, seed=11)
    c.table[0, 1] = c.kc.shape[0] + 9
    c.K[0][16:32] = 0
    c.V[0][16:32] = 0
    c.check(c.run(sv))
    c.table[0, 1] = -3
    c.check(c.run(sv))


def test_attention_offsets_past_32_bits(sv):
    """The last blocks of a cache of more than 2^32 entries (8.6 GB for each of K and V)."""
    Hk, bs, D = 8, 64, 128
    nb = (1 << 32) // (Hk * bs * D) + 40
    kc = torch.empty(nb, bs, Hk, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty(nb, bs, Hk, D, dtype=torch.bfloat16, device="cuda")
    c = Case([300], [5], 16, Hk, D, torch.bfloat16, bs, seed=12)
    n = c.kc.shape[0]
    kc[nb - n:] = c.kc
    vc[nb - n:] = c.vc
    c.kc, c.vc = kc, vc
    c.table = c.table + (nb - n)
    c.check(c.run(sv))
    # and the writers reach them
    x = torch.randn(2, Hk, D, device="cuda").to(torch.bfloat16)
    slot = torch.tensor([nb * bs - 1, 3], device="cuda")
    sv.rope_cache(x, x, x, _i32([0, 0]), slot, sv.rope_freqs(D), kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc[nb - 1, bs - 1], x[0]) and torch.equal(vc[nb - 1, bs - 1], x[0])


def test_attention_without_tokens_or_blocks(sv):
    """No packed token at all, no token that attends, and a table without a column."""
    c = Case([30, 7], [2, 1], 4, 2, 64, seed=16)
    status = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    none = torch.empty((0, 4, 64), dtype=c.dtype, device="cuda")
    sv.tree_attention(none, c.kc, c.vc, c.table, _i32(c.kv), _i32([0, 0, 0]), 0, out=dict(out=none, status=status))
    torch.cuda.synchronize()
    assert (status == 0).all()
    out = dict(out=torch.full_like(c.q, 5.0), status=status.fill_(-1))
    sv.tree_attention(c.q, c.kc, c.vc, c.table, _i32(c.kv), _i32(c.cu), 0, out=out)
    torch.cuda.synchronize()
    assert (out["out"] == 5).all() and (status == 0).all()
    got = sv.tree_attention(c.q, c.kc, c.vc, c.table[:, :0].contiguous(), _i32(c.kv), _i32(c.cu), 2, with_lse=True)
    torch.cuda.synchronize()
    assert (got["out"] == 0).all() and torch.isneginf(got["lse"]).all()


def test_attention_on_another_stream(sv):
    c = Case([900, 33], [9, 9], 8, 2, 128, seed=13)
    want = c.run(sv)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q = c.q * 1  # made on this stream
        got = sv.tree_attention(q, c.kc, c.vc, c.table, _i32(c.kv), _i32(c.cu), 9, scale=c.scale, with_lse=True)
    s.synchronize()
    assert torch.equal(got["out"], want["out"])


def test_attention_in_a_graph(sv):
    """The launches depend on host sizes alone: a captured step replays on new lengths."""
    c = Case([2000, 33], [9, 9], 8, 2, 128, seed=14)
    kv, cu = _i32(c.kv), _i32(c.cu)
    ws = torch.empty(sv.tree_attention_workspace(2, 18, 9, 8, 2, 128, c.table.shape[1] * 16), dtype=torch.uint8, device="cuda")
    out = dict(out=torch.empty_like(c.q), lse=torch.empty(18, 8, device="cuda"))
    call = lambda: sv.tree_attention(c.q, c.kc, c.vc, c.table, kv, cu, 9, scale=c.scale, out=out, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    kv.copy_(_i32([1111, 42]))
    g.replay()
    torch.cuda.synchronize()
    c.kv = [1111, 42]
    c.K[0], c.V[0] = c.K[0][:1111], c.V[0][:1111]
    c.check(out)


# --- commit ----------------------------------------------------------------------------------------------------
def _commit_case(R, branches, k, layers, Hk, D, bs, seed, path=None, dtype=torch.bfloat16, head_major=False):
    rng = np.random.default_rng(seed)
    n = 1 + branches * k
    seq = rng.integers(0, 100, R)
    new = np.full(R, n)
    new[rng.random(R) < 0.15] = 0
    kv = seq + new
    if R > 3:
        kv[1] = 0  # took no part
    mb = max(1, int(max(-(-(seq + n) // bs))))
    nb = int(sum(-(-x // bs) for x in kv)) + 10
    order = rng.permutation(nb).astype(np.int32)
    table = np.full((R, mb), -1, np.int32)
    at = 0
    for r in range(R):
        h = -(-int(kv[r]) // bs)
        table[r, :h] = order[at:at + h]
        at += h
    free = np.full(nb, -9, np.int32)
    free[:nb - at] = order[at:]
    shape = (layers, nb, Hk, bs, D) if head_major else (layers, nb, bs, Hk, D)
    g = torch.Generator(device="cuda").manual_seed(seed)
    kc, vc = (torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2))
    if head_major:
        kc, vc = kc.transpose(2, 3), vc.transpose(2, 3)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return dict(seq=seq, kv=kv, cu=cu, table=table, free=free, count=nb - at, kc=kc, vc=vc,
                accept=rng.integers(-1, k + 2, R).astype(np.int32), branch=rng.integers(0, branches, R).astype(np.int32))


def _check_commit(sv, c, k, branch=None, path=None):
    want = plain.commit(_np(c["kc"]), _np(c["vc"]), c["table"], c["seq"], c["kv"], c["cu"], c["accept"], k, c["free"],
                        c["count"], branch, path)
    free = _i32(c["free"])
    kc, vc = c["kc"], c["vc"]
    if kc.shape[0] == 1:
        kc, vc = kc[0], vc[0]
    got = sv.cache_commit(kc, vc, _i32(c["table"]), _i32(c["seq"]), _i32(c["kv"]), _i32(c["cu"]), _i32(c["accept"]), k,
                          free, _i32([c["count"]]), branch=None if branch is None else _i32(branch),
                          path=None if path is None else _i32(path))
    torch.cuda.synchronize()
    for name in ("seq_len", "free_count", "status"):
        _same(got[name], want[name], name)
    _same(free, want["free"], "free")
    np.testing.assert_array_equal(_np(c["kc"]), want["k"])
    np.testing.assert_array_equal(_np(c["vc"]), want["v"])
    return want


@pytest.mark.parametrize("R,branches,k,layers,Hk,D,bs", [
    (1, 2, 4, 1, 1, 8, 8), (6, 2, 32, 3, 4, 128, 16), (40, 8, 4, 2, 2, 64, 24), (3, 3, 0, 2, 2, 64, 16),
    (300, 2, 5, 1, 3, 40, 8), (5, 1, 30, 2, 16, 128, 64), (4, 3, 100, 2, 2, 72, 48)])
def test_commit_branches(sv, R, branches, k, layers, Hk, D, bs):
    c = _commit_case(R, branches, k, layers, Hk, D, bs, seed=R + k, head_major=R == 40)
    _check_commit(sv, c, k, branch=c["branch"])
    if branches == 1:
        c = _commit_case(R, branches, k, layers, Hk, D, bs, seed=R + k + 1)
        _check_commit(sv, c, k)


def test_commit_paths(sv):
    """Paths through arbitrary trees, sources and destinations interleaved; a path that falls or leaves the tree ends."""
    R, k, n = 50, 40, 81
    c = _commit_case(R, 2, k, 2, 2, 64, 16, seed=20)
    rng = np.random.default_rng(21)
    path = np.stack([np.sort(rng.choice(np.arange(1, n), k, replace=False)) for _ in range(R)]).astype(np.int32)
    path[0] = np.arange(1, k + 1)
    path[2] = np.arange(2, k + 2)
    path[5, 7] = path[5, 6]
    path[6, 3] = n + 4
    path[7, 0] = 0
    c["accept"][5:8] = k
    want = _check_commit(sv, c, k, path=path)
    assert (want["status"] == 512).any()


def test_commit_bad_branch(sv):
    c = _commit_case(4, 2, 4, 1, 2, 64, 16, seed=22)
    c["accept"][:] = 4
    c["branch"][:] = [-1, 0, 2, 1 << 30]
    _check_commit(sv, c, 4, branch=c["branch"])


# --- refusals --------------------------------------------------------------------------------------------------
def test_binding_refuses(sv):
    c = Case([20], [3], 4, 2, 64)
    i = _i32([0])

    def attn(**kw):
        a = dict(q=c.q, k=c.kc, v=c.vc, table=c.table, kv=_i32(c.kv), cu=_i32(c.cu))
        a.update(kw)
        return sv.tree_attention(a["q"], a["k"], a["v"], a["table"], a["kv"], a["cu"], 3)

    with pytest.raises(TypeError):
        attn(q=c.q.float())
    with pytest.raises(sv.SpecVerifyError) as e:
        attn(q=c.q.half())  # q and the cache in different types
    assert e.value.code == -2
    with pytest.raises(ValueError):
        attn(q=c.q.transpose(1, 2))
    with pytest.raises(ValueError):
        attn(kv=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        attn(cu=_i32([0, 1, 3]))
    with pytest.raises(ValueError):
        attn(v=c.vc.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3))  # other strides than K
    with pytest.raises(sv.SpecVerifyError) as e:
        attn(q=torch.zeros(3, 3, 64, dtype=torch.bfloat16, device="cuda"))  # heads no multiple of kv_heads
    assert e.value.code == -3
    with pytest.raises(sv.SpecVerifyError) as e:
        attn(q=torch.zeros(3, 4, 72, dtype=torch.bfloat16, device="cuda")[:, :, 4:68])  # 8-byte aligned heads
    assert e.value.code == -7
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.tree_attention(c.q, c.kc, c.vc, c.table, _i32(c.kv), _i32(c.cu), 3,
                          workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -6
    with pytest.raises(ValueError):
        sv.step_tables(i, i, i, i, i, 16, 4)  # a table of one dimension
    with pytest.raises(ValueError):
        sv.rope_cache(c.q, c.q[:, :2], c.q[:, :2], _i32([0, 1, 2]), _i32([0, 1, 2]), sv.rope_freqs(64), c.kc, c.vc)
    with pytest.raises(sv.SpecVerifyError) as e:  # more rotated entries than the head has
        sv.rope_cache(c.q, c.q[:, :2], c.q[:, :2], _i32([0, 1, 2]), torch.zeros(3, dtype=torch.int64, device="cuda"),
                      sv.rope_freqs(128), c.kc, c.vc)
    assert e.value.code == -3
