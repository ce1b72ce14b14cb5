"""norm_rope_cache on the GPU against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from tests import cache_plain, pages_plain as plain
from tests.test_gpu_cache import TINY, UNIT, _i32, _np, _rope_bound, _rope_case

pytestmark = pytest.mark.gpu

# Relative error of a normed entry in fp32, in units of 2^-24: a sum of at most 128 squares takes at most 16 fused
# steps and 5 exchanges (21), the mean, its constant and eps 3 more; the square root halves these 24.  rsqrtf is within
# 2 units in the last place (4); the weight's product and the entry's are a rounding each (2).
NORM = (24 / 2 + 4 + 2) * 2.0 ** -24


def _weights(kind, D, dtype, seed):
    if kind == "none":
        return None
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1 + torch.randn(D, generator=g, device="cuda")).to(dtype if kind == "own" else torch.float32)


def _check(sv, T, Hq, Hk, D, rot, interleaved, dtype, kind="own", eps=1e-6, fused=True, head_major=False, scale=1.0,
           mscale=1.0, one_of=None):
    q, k, v, kc, vc, slot = _rope_case(T, Hq, Hk, D, dtype, seed=T + D, fused=fused, head_major=head_major)
    q.mul_(scale), k.mul_(scale)
    rng = np.random.default_rng(T)
    pos = rng.integers(0, 131072, T).astype(np.int32)
    pos[0] = 0
    if T > 4:
        slot[2], slot[3] = -1, kc.shape[0] * kc.shape[1]  # neither is written
        q[1, 0], k[4, Hk - 1] = 0, 0
    freqs = sv.rope_freqs(rot, 10000.0)
    qw, kw = _weights(kind, D, dtype, 1), _weights(kind, D, dtype, 2)
    if one_of == "q":
        kw = None
    if one_of == "k":
        qw = None
    before = kc.clone()
    args = (_i32(pos), slot, freqs, kc, vc)
    named = dict(q_weight=qw, k_weight=kw, eps=eps, interleaved=interleaved, mscale=mscale)
    got = sv.norm_rope_cache(q, k, v, *args, **named)
    torch.cuda.synchronize()
    ang = cache_plain.turns(freqs.cpu().tolist(), pos)
    flat_k, flat_v = kc.reshape(-1, Hk, D), vc.reshape(-1, Hk, D)
    live = ((slot >= 0) & (slot < flat_k.shape[0])).cpu().numpy()
    for name, x, y, w in (("q", q, got, qw), ("k", k, flat_k[slot.clamp(0, flat_k.shape[0] - 1)], kw)):
        normed, want = plain.norm_rope(_np(x), None if w is None else _np(w), eps, ang, interleaved, mscale)
        half, pair = rot // 2, np.abs(normed) * NORM
        if half:  # both entries of a pair reach both results
            first = np.arange(half) * (2 if interleaved else 1)
            second = first + (1 if interleaved else half)
            pair[..., first] = pair[..., second] = abs(mscale) * (pair[..., first] + pair[..., second])
        tol = pair + _rope_bound(normed, half, mscale, dtype, interleaved)
        tol = tol + UNIT[dtype] * (np.abs(want) + tol) + TINY[dtype]
        err = np.abs(_np(y) - want)
        rows = live if name == "k" else slice(None)
        assert (err[rows] <= tol[rows]).all(), (name, (err / np.maximum(tol, 1e-300))[rows].max())
    lv = torch.from_numpy(live).cuda()
    assert torch.equal(flat_v[slot[lv]], v[lv])
    untouched = torch.ones(flat_k.shape[0], dtype=torch.bool, device="cuda")
    untouched[slot[lv]] = False
    assert torch.equal(flat_k[untouched], before.reshape(-1, Hk, D)[untouched])
    q2 = q.clone() if q.is_contiguous() else q
    same = sv.norm_rope_cache(q2, k, v, *args, **named, q_out=q2)
    torch.cuda.synchronize()
    assert torch.equal(same, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [
    (1, 1, 1, 8, 8), (1, 32, 8, 128, 128), (9, 28, 4, 128, 64), (65, 6, 3, 96, 96), (33, 5, 5, 80, 20),
    (17, 4, 2, 64, 0), (40, 8, 1, 72, 36), (300, 3, 3, 16, 2), (5, 64, 2, 128, 48), (7, 2, 1, 24, 24), (5000, 3, 1, 40, 32),
    (6, 1, 1, 16, 16), (6, 2, 2, 32, 32), (20000, 1, 1, 8, 0), (4863, 2, 1, 104, 64), (4864, 1, 2, 48, 48),
    (50, 4, 2, 128, 88), (50, 4, 2, 64, 40), (50, 4, 2, 120, 60), (50, 4, 2, 56, 44), (3000, 3, 1, 72, 72), (3000, 3, 1, 88, 46),
    (31, 2, 1, 8, 4), (31, 2, 1, 128, 4)])
def test_norm_rope(sv, T, Hq, Hk, D, rot, interleaved, dtype):
    _check(sv, T, Hq, Hk, D, rot, interleaved, dtype, kind=("own", "float", "none")[T % 3], fused=T != 65,
           head_major=T == 33, mscale=1.0 if T != 9 else 1.2772588722239782)


@pytest.mark.parametrize("kind", ["own", "float", "none"])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1.0])
@pytest.mark.parametrize("scale", [2.0 ** -10, 1.0, 2.0 ** 6])
def test_weights_and_sizes(sv, kind, eps, scale):
    if eps == 0.0:  # a head of zeros has no norm then: the next test's
        _check(sv, 4, 4, 2, 128, 128, False, torch.bfloat16, kind, eps, scale=scale)
    else:
        _check(sv, 30, 4, 2, 128, 128, False, torch.bfloat16, kind, eps, scale=scale)
        _check(sv, 30, 4, 2, 80, 20, False, torch.float16, kind, eps, scale=scale)


def test_one_weight_alone(sv):
    for one in "qk":
        _check(sv, 30, 4, 2, 128, 128, False, torch.bfloat16, "own", one_of=one)
        _check(sv, 30, 4, 2, 80, 20, False, torch.bfloat16, "float", one_of=one)


def test_zeros_and_no_numbers(sv):
    """A head of zeros without eps, and one with an infinity or NaN, is NaN throughout; its neighbours are not."""
    for D, rot in ((128, 128), (80, 20)):
        q, k, v, kc, vc, slot = _rope_case(6, 4, 2, D, torch.bfloat16)
        q[1, 2], q[2, 0, 3], k[4, 1, D - 1] = 0, float("nan"), float("nan")
        got = sv.norm_rope_cache(q, k, v, _i32([0] * 6), slot, sv.rope_freqs(rot), kc, vc, eps=0.0)
        bad = torch.isnan(got)
        assert bad[1, 2].all() and bad[2, 0].all() and bad.sum() == 2 * D
        bad = torch.isnan(kc.view(-1, 2, D)[slot])
        assert bad[4, 1].all() and bad.sum() == D


def test_heads_in_another_order(sv):
    """q with the heads in front: the result has the tokens in front, and the same values."""
    q, k, v, kc, vc, slot = _rope_case(30, 4, 2, 64, torch.bfloat16)
    args = (k, v, _i32(range(30)), slot, sv.rope_freqs(64), kc, vc)
    want = sv.norm_rope_cache(q, *args)
    got = sv.norm_rope_cache(q.transpose(0, 1).contiguous().transpose(0, 1), *args)
    assert got.is_contiguous() and torch.equal(got, want)


def test_the_norm_is_of_each_head_alone(sv):
    """Heads that differ by powers of two come out the same."""
    q, k, v, kc, vc, slot = _rope_case(40, 4, 2, 128, torch.bfloat16)
    base = torch.randn(40, 1, 128, device="cuda").bfloat16()
    q.copy_(base * 2.0 ** torch.arange(-4, 4, 2, device="cuda").view(1, 4, 1))
    got = sv.norm_rope_cache(q, k, v, _i32(range(40)), slot, sv.rope_freqs(128), kc, vc, eps=0.0)
    assert all(torch.equal(got[:, 0], got[:, h]) for h in range(1, 4))


def test_captured_and_replayed(sv):
    q, k, v, kc, vc, slot = _rope_case(9, 4, 2, 128, torch.bfloat16)
    args = (_i32(range(9)), slot, sv.rope_freqs(128), kc, vc)
    want = sv.norm_rope_cache(q, k, v, *args)
    wk = kc.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sv.norm_rope_cache(q, k, v, *args)
    got.zero_(), kc.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(kc.view(-1, 2, 128)[slot], wk.view(-1, 2, 128)[slot])


def test_refusals(sv):
    q, k, v, kc, vc, slot = _rope_case(3, 4, 2, 64, torch.bfloat16)
    w = torch.ones(64, device="cuda")
    args = (_i32([0, 1, 2]), slot, sv.rope_freqs(64), kc, vc)
    call = lambda **more: sv.norm_rope_cache(q, k, v, *args, **dict(dict(q_weight=w, k_weight=w), **more))  # noqa: E731
    call()
    for bad in (w[:63], w.cpu(), torch.ones(128, device="cuda")[::2]):
        for name in ("q_weight", "k_weight"):
            with pytest.raises(ValueError, match=name):
                call(**{name: bad})
    with pytest.raises(TypeError):
        call(q_weight=w.bfloat16())                       # two types
    with pytest.raises(TypeError):
        call(q_weight=w.double(), k_weight=w.double())
    with pytest.raises(sv.SpecVerifyError):
        call(q_weight=w.half(), k_weight=w.half())        # fp16 weights beside bf16 heads
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(sv.SpecVerifyError):
            call(eps=eps)
    with pytest.raises(ValueError, match="slot"):
        sv.norm_rope_cache(q, k, v, args[0], slot.int(), *args[2:])
    with pytest.raises(ValueError, match="freqs"):
        sv.norm_rope_cache(q, k, v, args[0], slot, args[2].cpu(), *args[3:])
    with pytest.raises(sv.SpecVerifyError):
        sv.norm_rope_cache(q, k.half(), v, *args)
    torch.cuda.synchronize()
