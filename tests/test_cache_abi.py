"""Argument checks and the frequency tables of the cache operators; nothing here touches a GPU."""
import ctypes as C
import math
import os
import shutil

import numpy as np
import pytest


@pytest.fixture(scope="module")
def m():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from serving_sampler_gb300 import _build

    _build.build()
    import serving_sampler_gb300 as sv

    sv.load()
    return sv


P = C.c_void_p
BUF, WS = P(0x10000), P(0x20000)


def _cache(m, **kw):
    a = dict(k=0x10000, v=0x20000, dtype=0, num_blocks=4, block_size=16, kv_heads=2, head_dim=64, layers=1,
             block_stride=2048, token_stride=128, head_stride=64, layer_stride=8192)
    a.update(kw)
    return m.SvKvCache(*a.values())


def _heads(m, heads=4, tokens=3, dim=64, dtype=0, data=0x10000, st=None, sh=None):
    return m.SvHeads(data, dtype, tokens, heads, dim, heads * dim if st is None else st, dim if sh is None else sh)


def test_step_tables_checks(m):
    f = m.load().sv_step_tables

    def call(R=2, bs=16, mb=4, nb=8, parent=None, T=6, words=0, seq=BUF, slot=BUF, mask=None, cu=BUF, pos=BUF):
        return f(seq, BUF, R, bs, BUF, mb, BUF, BUF, nb, parent, T, cu, BUF, slot, pos, mask, words, BUF, None, None)

    assert call(R=0) == 0
    assert call(R=-1) == -1 and call(bs=0) == -1 and call(mb=-1) == -1 and call(nb=-1) == -1 and call(T=-1) == -1
    assert call(words=-1) == -1
    assert call(parent=BUF, words=0) == -1           # parents ask for a mask
    assert call(parent=BUF, words=1, mask=None) == -1
    assert call(mb=1 << 28, bs=16) == -4             # positions past 2^31
    assert call(seq=None) == -1 and call(slot=None) == -1 and call(cu=None) == -1 and call(pos=None) == -1
    assert call(slot=P(0x10004)) == -7               # 8-byte entries
    assert call(seq=P(0x10002)) == -7


def test_cache_and_head_checks(m):
    lib = m.load()
    f = lib.sv_tree_attention

    def call(cache=None, q=None, out=None, R=1, mb=4, mt=3, mask=None, words=0, ws=WS, nbytes=1 << 40, kv=BUF, table=BUF):
        q = q or _heads(m)
        return f(q, cache or _cache(m), table, mb, kv, BUF, R, mt, mask, words, 1.0, out or q, None, None, ws, nbytes, None)

    assert call(R=0) == 0 and call(q=_heads(m, tokens=0)) == 0
    assert call(R=-1) == -1 and call(mb=-1) == -1 and call(mt=-1) == -1 and call(words=-1) == -1
    assert call(mask=BUF, words=0) == -1
    assert call(cache=_cache(m, dtype=1)) == -2       # fp32 caches are not taken
    assert call(q=_heads(m, dtype=2)) == -2           # q in another type than the cache
    assert call(cache=_cache(m, head_dim=60)) == -3 and call(cache=_cache(m, block_size=12)) == -3
    assert call(cache=_cache(m, head_dim=136)) == -4
    assert call(cache=_cache(m, layers=2)) == -3
    assert call(cache=_cache(m, token_stride=32)) == -3 and call(cache=_cache(m, head_stride=8)) == -3
    assert call(cache=_cache(m, block_stride=-2048)) == -3
    assert call(cache=_cache(m, token_stride=132)) == -7 and call(cache=_cache(m, k=0x10008)) == -7
    assert call(cache=_cache(m, v=None)) == -1
    assert call(q=_heads(m, heads=3)) == -3           # no multiple of kv_heads
    assert call(q=_heads(m, heads=512)) == -4         # more than SV_MAX_GROUP to a key head
    assert call(q=_heads(m, dim=72)) == -3
    assert call(q=_heads(m, data=0x10008)) == -7 and call(q=_heads(m, st=260)) == -7
    assert call(q=_heads(m, st=8)) == -3 and call(q=_heads(m, sh=8)) == -3
    assert call(out=_heads(m, heads=2)) == -3 and call(out=_heads(m, tokens=2)) == -3
    assert call(kv=None) == -1 and call(table=None) == -1 and call(kv=P(0x10002)) == -7
    assert call(mb=1 << 28) == -4
    assert call(ws=None) == -6 and call(nbytes=8) == -6 and call(ws=P(0x20010)) == -6
    size = lib.sv_tree_attention_workspace
    assert size(1, 3, 3, 4, 2, 64, 64) > 0
    assert size(-1, 3, 3, 4, 2, 64, 64) == 0 and size(1, 3, 3, 3, 2, 64, 64) == 0 and size(1, 3, 3, 4, 2, 136, 64) == 0
    assert size(1, 3, 3, 512, 2, 64, 64) == 0 and size(1, 3, 3, 4, 2, 64, 1 << 31) == 0


def test_rope_checks(m):
    f = m.load().sv_rope_cache

    def call(q=None, k=None, v=None, rot=64, inter=0, cache=None, pos=BUF, slot=BUF, freqs=BUF, out=None):
        q = q or _heads(m)
        k = k or _heads(m, heads=2)
        return f(q, k, v or k, pos, slot, freqs, rot, inter, 1.0, out or q, cache or _cache(m), None)

    empty = _heads(m, tokens=0)
    assert call(q=empty, k=_heads(m, heads=2, tokens=0)) == 0
    assert call(inter=2) == -1
    assert call(rot=66) == -3 and call(rot=7) == -3 and call(rot=-2) == -3
    assert call(k=_heads(m, heads=3)) == -3 and call(k=_heads(m, heads=2, tokens=2)) == -3
    assert call(v=_heads(m, heads=1)) == -3
    assert call(out=_heads(m, heads=5)) == -3 and call(out=_heads(m, dtype=2)) == -2
    assert call(pos=None) == -1 and call(slot=None) == -1 and call(freqs=None) == -1
    assert call(slot=P(0x10004)) == -7 and call(freqs=P(0x10004)) == -7
    assert call(cache=_cache(m, layers=3)) == -3


def test_commit_checks(m):
    f = m.load().sv_cache_commit

    def call(cache=None, R=2, branch=None, path=None, k=4, mb=4, accept=BUF, free=BUF, seq_out=BUF):
        return f(cache or _cache(m), BUF, mb, BUF, BUF, BUF, R, accept, branch, path, k, free, BUF, seq_out, BUF, None, None)

    assert call(R=0) == 0
    assert call(R=-1) == -1 and call(k=-1) == -1 and call(mb=-1) == -1
    assert call(k=257) == -4
    assert call(branch=BUF, path=BUF) == -1
    assert call(cache=_cache(m, layers=600000)) == -4
    assert call(cache=_cache(m, layers=2, layer_stride=4)) == -3
    assert call(accept=None) == -1 and call(free=None) == -1 and call(seq_out=None) == -1
    assert call(branch=P(0x10002)) == -7


def test_valid_calls_without_a_device(m):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    lib = m.load()
    q, k = _heads(m), _heads(m, heads=2)
    assert lib.sv_rope_cache(q, k, k, BUF, BUF, BUF, 64, 0, 1.0, q, _cache(m), None) == -8
    assert lib.sv_cache_commit(_cache(m), BUF, 4, BUF, BUF, BUF, 2, BUF, None, None, 4, BUF, BUF, BUF, BUF, None, None) == -8


def _freqs(m, *a):
    return [int(x) % (1 << 64) for x in m.rope_freqs(*a, device="cpu").tolist()]


def _close(got, inv_freq):
    """Turn fractions: equal up to fp64's rounding of the frequency, around the circle."""
    for g, f in zip(got, inv_freq):
        want = (f / (2 * math.pi)) % 1.0
        d = abs(g / 2.0 ** 64 - want)
        assert min(d, 1 - d) <= 2.0 ** -50, (g, f)


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (128, 10000.0), (64, 500000.0), (96, 1e6), (0, 10.0)])
def test_rope_frequencies(m, rot, base):
    half = rot // 2
    inv = [base ** (-i / half) for i in range(half)]
    got = _freqs(m, rot, base)
    assert len(got) == half
    _close(got, inv)
    _close(_freqs(m, rot, base, m.ROPE_LINEAR, 4.0), [f / 4 for f in inv])
    if rot > 2:
        b = base * 8.0 ** (rot / (rot - 2))
        _close(_freqs(m, rot, base, m.ROPE_BASE, 8.0), [b ** (-i / half) for i in range(half)])


def test_rope_scaled_by_parts(m):
    rot, base, factor, trained, low, high = 128, 10000.0, 16.0, 4096.0, 1.0, 32.0
    half = rot // 2
    inv = np.array([base ** (-i / half) for i in range(half)])
    turns = trained * inv / (2 * math.pi)
    keep = np.clip((turns - low) / (high - low), 0, 1)
    got = _freqs(m, rot, base, m.ROPE_BY_TURNS, factor, trained, low, high)
    _close(got, inv * keep + inv / factor * (1 - keep))
    assert keep[0] == 1 and keep[-1] == 0
    # by the pair's index: the ends of the ramp are the pairs that turn `high` and `low` times
    first = math.floor(half * math.log(trained / (high * 2 * math.pi)) / math.log(base))
    last = math.ceil(half * math.log(trained / (low * 2 * math.pi)) / math.log(base))
    keep = 1 - np.clip((np.arange(half) - first) / (last - first), 0, 1)
    got = _freqs(m, rot, base, m.ROPE_BY_DIM, factor, trained, low, high)
    _close(got, inv * keep + inv / factor * (1 - keep))


def test_rope_frequency_checks(m):
    f = m.load().sv_rope_freqs
    assert f(7, 1e4, 0, 1, 0, 0, 0, BUF) == -1 and f(-2, 1e4, 0, 1, 0, 0, 0, BUF) == -1
    assert f(8, 0.0, 0, 1, 0, 0, 0, BUF) == -1 and f(8, float("nan"), 0, 1, 0, 0, 0, BUF) == -1
    assert f(8, 1e4, 5, 1, 0, 0, 0, BUF) == -1 and f(8, 1e4, 1, 0.0, 0, 0, 0, BUF) == -1
    assert f(8, 1e4, 3, 4.0, 4096.0, 32.0, 1.0, BUF) == -1 and f(8, 1e4, 4, 4.0, 0.0, 1.0, 32.0, BUF) == -1
    assert f(2, 1e4, 2, 4.0, 0, 0, 0, BUF) == -3
    assert f(8, 1e4, 0, 1, 0, 0, 0, None) == -1 and f(8, 1e4, 0, 1, 0, 0, 0, P(0x10004)) == -7
    assert f(0, 1e4, 0, 1, 0, 0, 0, None) == 0


@pytest.mark.parametrize("kv_heads", [1, 2, 8, 60, 200])
@pytest.mark.parametrize("tokens", [1, 300])
def test_attention_workspace_holds_every_group(m, kv_heads, tokens):
    """Room for all but the first group of an item in every CTA, when many requests make the shares long."""
    sms, D = 152, 128  # what the library takes where there is no device
    rows = 256 if tokens > 128 else 8
    per_head = -(-(-(-tokens // 128)) // 2)
    for keys in (1000, 131072, 1 << 20, 20_000_000, 1 << 30):
        nt = -(-keys // 128)
        wave = max(1, sms // (kv_heads * per_head))
        root, one, two = 2 * int(0.75 * nt ** 0.5), -(-nt // wave), -(-nt // (2 * wave))
        even = two if 5 * two >= 4 * root else one if 5 * one >= 4 * root else root
        size = (max(8 if tokens > 128 else 2, even) + 1) // 2 * 2
        groups = -(-nt // size)
        got = m.tree_attention_workspace(100_000, 100_000 * tokens, tokens, kv_heads, kv_heads, D, keys)
        assert got >= sms * groups * rows * (D + 2) * 4, keys
