"""Cases for the operators around a paged key/value cache in a speculative verify step.

  tables  step_tables: blocks, slots, positions and ancestor masks of a step's tokens from lengths and parents
  rope    rope_cache: rotary positions on q and k, k and v written into their cache slots
  attn    tree_attention: attention of a tree (or chain) of drafted tokens over the paged cache
  commit  cache_commit: the accepted path's keys and values moved behind the committed ones, blocks given back

A request's tokens of one step are its last committed token (the root) and `branches` drafts of `k` tokens that
hang from it, 1 + branches * k in all.  `run` computes an operator in elementary torch operations, or calls the
package's own entry points where `own` is true.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _tables(name, R, branches, k, lo, hi, block):
    return dict(name=name, op="tables", R=R, branches=branches, k=k, lo=lo, hi=hi, block=block)


def _rope(name, R, branches, k, lo, hi, heads, kv_heads, dim, rot, interleaved, scaling, block, dtype):
    return dict(name=name, op="rope", R=R, branches=branches, k=k, lo=lo, hi=hi, heads=heads, kv_heads=kv_heads, dim=dim,
                rot=rot, interleaved=interleaved, scaling=scaling, block=block, dtype=dtype)


def _attn(name, R, branches, k, lo, hi, group, kv_heads, dim, block, dtype, tree):
    return dict(name=name, op="attn", R=R, branches=branches, k=k, lo=lo, hi=hi, group=group, kv_heads=kv_heads, dim=dim,
                block=block, dtype=dtype, tree=tree)


def _commit(name, R, branches, k, lo, hi, layers, kv_heads, dim, block, dtype):
    return dict(name=name, op="commit", R=R, branches=branches, k=k, lo=lo, hi=hi, layers=layers, kv_heads=kv_heads,
                dim=dim, block=block, dtype=dtype)


def listed():
    return [
        # one request verifying a chain of 8 drafts: the per-step bookkeeping of an interactive session
        _tables("tables-1x9", 1, 1, 8, 1000, 1000, 16),
        # the throughput sweep's largest batch, every request with two branches of 32 drafts
        _tables("tables-1024x65", 1024, 2, 32, 100, 6000, 16),
        # one request's chain in one layer
        _rope("rope-1x9", 1, 1, 8, 1000, 1000, 32, 8, 128, 128, False, "none", 16, "bf16"),
        # 64 listening sessions, a main draft and a runner-up of 32 tokens, half of each head rotated, pairs side by side
        _rope("rope-64x65", 64, 2, 32, 500, 4000, 28, 4, 128, 64, True, "none", 64, "bf16"),
        # long draft chains past the trained positions, frequencies scaled by parts, a head size that is no power of two
        _rope("rope-60x257", 60, 1, 256, 1000, 9000, 32, 8, 96, 96, False, "parts", 32, "fp16"),
        # a single token of a single request over a short cache: the plain decode step
        _attn("attn-1x1", 1, 1, 0, 777, 777, 4, 8, 128, 16, "bf16", False),
        # a serving batch verifying chains of 8 drafts
        _attn("attn-64x9", 64, 1, 8, 500, 8000, 4, 8, 128, 16, "bf16", False),
        # listening sessions: two branches of 32 drafts, seven query heads to a key head
        _attn("attn-64x65", 64, 2, 32, 1000, 4000, 7, 4, 128, 64, "bf16", True),
        # 17 requests with bushy trees, every query head with its own key head, half precision, a block that is no power of two
        _attn("attn-17x33", 17, 8, 4, 333, 3001, 1, 16, 64, 48, "fp16", True),
        # one chain over a very long context
        _attn("attn-1x9-131071", 1, 1, 8, 131071, 131071, 4, 8, 128, 16, "bf16", False),
        # a small batch after verification, a few layers' cache
        _commit("commit-4x9", 4, 2, 4, 50, 90, 4, 8, 128, 16, "bf16"),
        # listening sessions after verification, the caches of 16 layers
        _commit("commit-64x65", 64, 2, 32, 20, 300, 16, 4, 128, 64, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rope", "attn", "attn", "attn", "commit"])
    branches = rng.choice([1, 1, 2, 3, 5, 8])
    block = rng.choice([8, 16, 16, 24, 32, 48, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "tables":
        R, k = _log(rng, 1, 1024), _log(rng, 1, 32)
        while R * (1 + branches * k) > 1024 * 65:
            R = max(1, R // 2)
        hi = _log(rng, 2, 6000)
        return _drop(_tables("", R, branches, k, rng.randint(0, hi), hi, block))
    dim = rng.choice([64, 80, 96, 128, 128, rng.randrange(8, 129, 8)])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
    if op == "rope":
        R, k = _log(rng, 1, 64), _log(rng, 1, 256 // branches)
        group = rng.choice([1, 2, 4, 5, 7, 8])
        while R * (1 + branches * k) * kv_heads * (group + 2) * dim > 60 * 257 * 48 * 96:
            R, k = max(1, R // 2), max(1, k - 1)
        rot = min(dim, rng.choice([dim, dim, dim // 2, max(2, dim // 4 * 2)]) // 2 * 2)
        hi = _log(rng, 2, 131000)
        hi = min(hi, max(2, 2_000_000 // (R * kv_heads)))
        return _drop(_rope("", R, branches, k, rng.randint(0, hi), hi, kv_heads * group, kv_heads, dim, rot,
                           rng.random() < 0.5, rng.choice(["none", "linear", "parts"]), block, dtype))
    if op == "commit":
        branches = max(2, branches)
        R, k, layers = _log(rng, 1, 64), _log(rng, 1, 32), _log(rng, 1, 16)
        hi = _log(rng, 2, 300)
        while R * (hi + branches * k + block) * layers * kv_heads * dim > 64 * 365 * 16 * 4 * 128:
            R, layers = max(1, R // 2), max(1, layers - 1)
        return _drop(_commit("", R, branches, k, rng.randint(0, hi), hi, layers, kv_heads, dim, block, dtype))
    R, group = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16])
    k = rng.choice([0, _log(rng, 1, 32), _log(rng, 1, 32), _log(rng, 1, 64)])
    k = min(k, 128 // branches)
    hi = _log(rng, 1, 131071)
    n = 1 + branches * k
    while R * kv_heads * (hi + n) * 128 > 64 * 8 * 8009 * 128 or R * kv_heads * group * n * (hi + n) > 64 * 28 * 65 * 4065:
        R, hi = max(1, R - 1 - R // 4), max(1, hi - hi // 8)
    return _drop(_attn("", R, branches, k, rng.randint(0, hi), hi, group, kv_heads, dim, block, dtype,
                       branches > 1 or rng.random() < 0.5))


def _drop(case):
    case.pop("name")
    return case


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _lengths(case):
    """Committed tokens of each request: the ends of the range and values between, a part of the case."""
    rng = random.Random(case["R"] * 1000003 + case["lo"] * 1009 + case["hi"])
    got = [case["hi"], case["lo"]] + [rng.randint(case["lo"], case["hi"]) for _ in range(case["R"])]
    return got[: case["R"]]


def _tokens(case):
    return 1 + case["branches"] * case["k"]


def _up(a, b):
    return -(-a // b)


def _parents(case):
    """Parent of each of a request's tokens: branch b is 1 + b k ... b k + k, its first token hangs from the root."""
    one = [-1]
    for b in range(case["branches"]):
        one += [0 if j == 0 else b * case["k"] + j for j in range(case["k"])]
    return one


def _paged(case, g, extra):
    """Block tables over a shuffled pool: every request holds the blocks of its length + `extra` tokens; the rest is free."""
    R, b = case["R"], case["block"]
    L = _lengths(case)
    n = _tokens(case)
    held = [_up(x + extra, b) for x in L]
    most = max(_up(x + n, b) for x in L)
    blocks = sum(_up(x + n, b) for x in L) + R + 3
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((R, most), -1, dtype=torch.int32, device="cuda")
    inside = torch.arange(most, device="cuda").view(1, -1) < torch.tensor(held, device="cuda").view(-1, 1)
    table[inside] = order[: sum(held)]
    free = torch.full((blocks,), -1, dtype=torch.int32, device="cuda")
    left = blocks - sum(held)
    free[:left] = order[sum(held):]
    return dict(table=table, blocks=blocks, free=free, free_count=torch.tensor([left], dtype=torch.int32, device="cuda"),
                seq_len=torch.tensor(L, dtype=torch.int32, device="cuda"), most=most)


def _freqs(case):
    """Turns per position of each pair as 64-bit fractions: 2^64 inv_freq / (2 pi)."""
    half = case["rot"] // 2
    out = []
    for i in range(half):
        f = 10000.0 ** (-i / half)
        if case["scaling"] == "linear":
            f /= 4.0
        elif case["scaling"] == "parts":  # pairs with few turns in the trained 8192 positions are stretched 16 times
            turns = 8192 * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
            f = f / 16.0 * (1 - keep) + f * keep
        x = int(round(f / (2 * math.pi) * 2.0 ** 64))
        out.append(x - 2 ** 64 if x >= 2 ** 63 else x)
    return torch.tensor(out, dtype=torch.int64, device="cuda")


def _visible_bits(case):
    """Host ancestor masks as 32-bit words [n, words] of a request's tokens (each sees itself and its ancestors)."""
    par, rows = _parents(case), []
    words = _up(len(par), 32)
    for j, p in enumerate(par):
        rows.append((rows[p] if p >= 0 else 0) | (1 << j))
    def word(m, w):
        x = (m >> (32 * w)) & 0xFFFFFFFF
        return x - 2 ** 32 if x >= 2 ** 31 else x
    return [[word(m, w) for w in range(words)] for m in rows]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    R, n = case["R"], _tokens(case)
    T = R * n
    s = dict(case=case, R=R, n=n, T=T, block=case["block"])
    cu = torch.arange(R + 1, dtype=torch.int32, device="cuda") * n
    if case["op"] == "tables":
        s.update(_paged(case, g, 0))
        s.update(new_len=torch.full((R,), n, dtype=torch.int32, device="cuda"), words=_up(n, 32),
                 parent=torch.tensor(_parents(case), dtype=torch.int32, device="cuda").repeat(R))
        return s
    dt, D, H = DTYPES[case["dtype"]], case["dim"], case["kv_heads"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)

    s.update(_paged(case, g, n))
    L = _lengths(case)
    s["kv_len"] = s["seq_len"] + n
    if case["op"] == "commit":
        shape = (case["layers"], s["blocks"], case["block"], H, D)
        a = torch.randint(0, case["k"] + 1, (R,), generator=g, device="cuda", dtype=torch.int32)
        b = torch.randint(0, case["branches"], (R,), generator=g, device="cuda", dtype=torch.int32)
        s.update(kc=randn(*shape), vc=randn(*shape), cu=cu, accept_len=a, branch=b, k=case["k"])
        return s
    shape = (s["blocks"], case["block"], H, D)
    if case["op"] == "rope":
        Hq = case["heads"]
        pos = torch.tensor(_parents(case), device="cuda")
        depth = torch.arange(n, device="cuda")
        depth = torch.where(depth > 0, (depth - 1) % max(1, case["k"]) + 1, depth)
        base = torch.arange(n, device="cuda").view(1, n) + s["seq_len"].view(R, 1)
        slot = s["table"].long().gather(1, base // case["block"]) * case["block"] + base % case["block"]
        qkv = randn(T, Hq + 2 * H, D)  # one projection's output; q, k and v are views of it
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + H], v=qkv[:, Hq + H:], slot=slot.reshape(T).contiguous(),
                 position=(s["seq_len"].view(R, 1) + depth).reshape(T).to(torch.int32).contiguous(),
                 freqs=_freqs(case), kc=torch.zeros(shape, dtype=dt, device="cuda"),
                 vc=torch.zeros(shape, dtype=dt, device="cuda"), interleaved=case["interleaved"],
                 mscale=1.0 if case["scaling"] != "parts" else 0.1 * math.log(16.0) + 1.0)
        return s
    s.update(kc=randn(*shape), vc=randn(*shape), cu=cu, G=case["group"], scale=1.0 / math.sqrt(D),
             q=randn(T, H * case["group"], D) * 2, most_kv=max(L) + n, mask=None)
    if case["tree"]:
        s["mask"] = torch.tensor(_visible_bits(case), dtype=torch.int32, device="cuda").repeat(R, 1)
    return s


# ---------------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------------
def _plain_tables(s):
    b, R, T = s["block"], s["R"], s["T"]
    L, new = s["seq_len"].long(), s["new_len"].long()
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), new.cumsum(0)])
    held, want = (L + b - 1) // b, (L + new + b - 1) // b
    need = want - held
    pre = need.cumsum(0) - need
    count = s["free_count"].long()
    fits = (need == 0) | (pre + need <= count)
    cols = torch.arange(s["most"], device="cuda").view(1, -1)
    i = pre.view(-1, 1) + cols - held.view(-1, 1)
    fresh = (cols >= held.view(-1, 1)) & (cols < want.view(-1, 1)) & fits.view(-1, 1)
    table = torch.where(fresh, s["free"][(count - 1 - i).clamp(0, s["blocks"] - 1)], s["table"])
    t = torch.arange(T, device="cuda")
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=R - 1)
    j = t - cu[r]
    at = L[r] + j
    slot = table[r, (at // b).clamp(max=s["most"] - 1)].long() * b + at % b
    slot = torch.where(fits[r], slot, -1)
    # ancestors: j sees x where x is reached from j by following parents; log2 steps double the reach
    n = s["n"]
    par = s["parent"].view(R, n)
    tree = (par.unsqueeze(2) == torch.arange(n, device="cuda")) | torch.eye(n, dtype=torch.bool, device="cuda")
    reach = tree.to(torch.float32)
    for _ in range(max(1, n - 1).bit_length()):
        reach = (reach @ reach > 0).to(torch.float32)
    position = L.view(R, 1) + reach.sum(2).long() - 1
    bits = torch.nn.functional.pad(reach, (0, s["words"] * 32 - n)).view(R * n, s["words"], 32).long()
    mask = (bits << torch.arange(32, device="cuda")).sum(2)
    mask = torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask)
    return dict(cu_tokens=cu.int(), kv_len=torch.where(fits, L + new, 0).int(), slot=slot, position=position.view(T).int(),
                mask=mask.int(), block_table=table, free_count=(count - (need * fits).sum()).int(),
                status=torch.where(fits, 0, 256).int())


def _plain_rotate(x, c, sn, interleaved):
    rot = 2 * c.shape[-1]
    x = x.float()
    a, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        u, w = a[..., 0::2], a[..., 1::2]
        y = torch.stack([u * c - w * sn, u * sn + w * c], -1).flatten(-2)
    else:
        u, w = a[..., : rot // 2], a[..., rot // 2:]
        y = torch.cat([u * c - w * sn, u * sn + w * c], -1)
    return torch.cat([y, rest], -1)


def _plain_rope(s):
    phase = s["position"].long().view(-1, 1) * s["freqs"].view(1, -1)  # wraps: whole turns drop out
    angle = (phase >> 32).float() * (2 * math.pi / 2.0 ** 32)
    c, sn = (torch.cos(angle) * s["mscale"]).unsqueeze(1), (torch.sin(angle) * s["mscale"]).unsqueeze(1)
    q = _plain_rotate(s["q"], c, sn, s["interleaved"]).to(s["q"].dtype)
    k = _plain_rotate(s["k"], c, sn, s["interleaved"]).to(s["k"].dtype)
    s["kc"].view(-1, *s["kc"].shape[2:])[s["slot"]] = k
    s["vc"].view(-1, *s["vc"].shape[2:])[s["slot"]] = s["v"]
    return dict(q=q, k_cache=s["kc"], v_cache=s["vc"])


def _plain_attn(s):
    R, n, G, b, most = s["R"], s["n"], s["G"], s["block"], s["most_kv"]
    H, D = s["kc"].shape[2:]
    x = torch.arange(most, device="cuda")
    at = s["table"].long().clamp(min=0)[:, x // b] * b + x % b  # [R, most]
    K = s["kc"].view(-1, H, D)[at].float().permute(0, 2, 3, 1)  # [R, H, D, most]
    Q = s["q"].view(R, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(R, H, n * G, D).float()
    S = (Q @ K) * s["scale"]
    del K
    rel = x.view(1, -1) - (s["kv_len"].long() - n).view(R, 1)  # drafted key index of each position
    j = torch.arange(n, device="cuda").view(1, n, 1)
    if s["mask"] is None:
        new = rel.view(R, 1, most) <= j
    else:
        word = (rel.clamp(0, n - 1) // 32).view(R, 1, most).expand(R, n, most)
        new = (s["mask"].view(R, n, -1).gather(2, word) >> (rel.clamp(min=0) % 32).view(R, 1, most)) & 1 > 0
    see = (rel.view(R, 1, most) < 0) | (new & (rel < n).view(R, 1, most))
    see = see.view(R, 1, n, 1, most)
    S = S.view(R, H, n, G, most).masked_fill_(~see, -math.inf)
    top = S.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    P = torch.exp(S - top).view(R, H, n * G, most)
    del S
    tot = P.sum(-1, keepdim=True)
    V = s["vc"].view(-1, H, D)[at].float().permute(0, 2, 1, 3)
    O = torch.where(tot > 0, (P @ V) / tot, 0.0)
    lse = top.view(R, H, n, G) + torch.log(tot).view(R, H, n, G)
    out = O.view(R, H, n, G, D).permute(0, 2, 1, 3, 4).reshape(R * n, H * G, D).to(s["q"].dtype)
    return dict(out=out, lse=lse.permute(0, 2, 1, 3).reshape(R * n, H * G))


def _plain_commit(s):
    b, R, n, k = s["block"], s["R"], s["n"], s["k"]
    L, a = s["seq_len"].long(), s["accept_len"].long().clamp(0, k)
    j = torch.arange(k, device="cuda").view(1, k)
    move = j < a.view(R, 1)
    src = L.view(R, 1) + 1 + s["branch"].long().view(R, 1) * k + j
    dst = L.view(R, 1) + 1 + j
    table = s["table"].long()
    width = table.shape[1] * b
    src, dst = (table.gather(1, x.clamp(max=width - 1) // b) * b + x % b for x in (src, dst))
    src, dst = src[move], dst[move]
    for c in (s["kc"], s["vc"]):
        flat = c.view(c.shape[0], -1, *c.shape[3:])
        flat[:, dst] = flat[:, src]
    new = L + 1 + a
    keep, held = (new + b - 1) // b, (s["kv_len"].long() + b - 1) // b
    give = held - keep
    pre = give.cumsum(0) - give
    cols = torch.arange(table.shape[1], device="cuda").view(1, -1)
    out = (cols >= keep.view(R, 1)) & (cols < held.view(R, 1))
    to = (s["free_count"].long() + pre.view(R, 1) + cols - keep.view(R, 1))[out]
    s["free"][to] = s["table"][out]
    return dict(k_cache=s["kc"], v_cache=s["vc"], seq_len=new.int(), free_blocks=s["free"],
                free_count=(s["free_count"] + give.sum()).int(), status=torch.zeros(R, dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"tables": _plain_tables, "rope": _plain_rope, "attn": _plain_attn, "commit": _plain_commit}[op](state)
    import serving_sampler_gb300 as sv

    s = state
    if op == "tables":
        got = sv.step_tables(s["seq_len"], s["new_len"], s["table"], s["free"], s["free_count"], s["block"], s["T"],
                             parent=s["parent"], mask_words=s["words"])
        return dict(got, block_table=s["table"])
    if op == "rope":
        q = sv.rope_cache(s["q"], s["k"], s["v"], s["position"], s["slot"], s["freqs"], s["kc"], s["vc"],
                          interleaved=s["interleaved"], mscale=s["mscale"])
        return dict(q=q, k_cache=s["kc"], v_cache=s["vc"])
    if op == "attn":
        if "workspace" not in s:  # kept by the program and shared by its layers
            nbytes = sv.tree_attention_workspace(s["R"], s["T"], s["n"], s["kc"].shape[2] * s["G"], s["kc"].shape[2],
                                                 s["kc"].shape[3], s["table"].shape[1] * s["block"])
            s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        return sv.tree_attention(s["q"], s["kc"], s["vc"], s["table"], s["kv_len"], s["cu"], s["n"], mask=s["mask"],
                                 scale=s["scale"], with_lse=True, workspace=s["workspace"])
    got = sv.cache_commit(s["kc"], s["vc"], s["table"], s["seq_len"], s["kv_len"], s["cu"], s["accept_len"], s["k"],
                          s["free"], s["free_count"], branch=s["branch"])
    return dict(got, k_cache=s["kc"], v_cache=s["vc"], free_blocks=s["free"])


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    R, n, b = case["R"], _tokens(case), case["block"]
    T, L = R * n, _lengths(case)
    if case["op"] == "tables":
        fresh = sum(_up(x + n, b) - _up(x, b) for x in L)
        touched = sum(_up(x + n, b) - x // b for x in L)
        words = _up(n, 32)
        return dict(bytes=8 * R + 4 * T + 4 * touched + 4 * fresh + 4 * (R + 1) + 8 * R + 12 * T + 4 * T * words + 8,
                    flops=float(T * words))
    D, H = case["dim"], case["kv_heads"]
    if case["op"] == "rope":
        rows = case["heads"] + 2 * H
        return dict(bytes=2 * 2 * T * rows * D + 12 * T + 4 * case["rot"],
                    flops=3.0 * T * (case["heads"] + H) * case["rot"] + 40.0 * T * case["rot"] / 2)
    if case["op"] == "attn":
        keys = sum(L) + R * n
        see = sum(bin(w & 0xFFFFFFFF).count("1") for row in _visible_bits(case) for w in row) if case["tree"] else n * (n + 1) // 2
        G = case["group"]
        bytes_ = 2 * keys * H * D * 2 + 2 * T * H * G * D * 2 + 4 * T * H * G + 4 * sum(_up(x + n, b) for x in L) + 8 * R
        if case["tree"]:
            bytes_ += 4 * T * _up(n, 32)
        return dict(bytes=bytes_, flops=4.0 * D * H * G * (sum(L) * n + R * see))
    # half of the drafts of a request are accepted on average; those of the first branch stay where they are
    moved = R * case["k"] / 2 * (case["branches"] - 1) / case["branches"]
    return dict(bytes=2 * 2 * 2 * moved * case["layers"] * H * D + 28 * R, flops=float(R))


# ---------------------------------------------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    L, b, n, R = _lengths(case), case["block"], s["n"], s["R"]
    table = s["table"].tolist()
    if case["op"] == "rope":
        pos = [L[r] + (0 if j == 0 else (j - 1) % case["k"] + 1) for r in range(R) for j in range(n)]
        turns = [int(x) % 2 ** 64 for x in s["freqs"].tolist()]
        half = case["rot"] // 2
        ang = torch.tensor([[(p * f % 2 ** 64) / 2.0 ** 64 for f in turns] for p in sorted(set(pos))], dtype=torch.float64)
        row = {p: i for i, p in enumerate(sorted(set(pos)))}
        ang = (ang * (2 * math.pi)).cuda()[torch.tensor([row[p] for p in pos], device="cuda")]
        first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        done = []
        for x in (s["q"], s["k"]):
            y = x.double()
            u, w = y[:, :, first].clone(), y[:, :, second].clone()
            turn = torch.polar(torch.full_like(ang, s["mscale"]), ang).unsqueeze(1) * torch.complex(u, w)
            y[:, :, first], y[:, :, second] = turn.real, turn.imag
            done.append(y)
        kc, vc = s["kc"].double(), s["vc"].double()
        for r in range(R):
            for j in range(n):
                at = L[r] + j
                kc[table[r][at // b], at % b] = done[1][r * n + j]
                vc[table[r][at // b], at % b] = s["v"][r * n + j].double()
        return dict(q=done[0], k_cache=kc, v_cache=vc)
    if case["op"] == "commit":
        kc, vc = s["kc"].double(), s["vc"].double()
        a, br = s["accept_len"].tolist(), s["branch"].tolist()
        for c in (kc, vc):
            for r in range(R):
                for j in range(a[r]):
                    src, dst = L[r] + 1 + br[r] * case["k"] + j, L[r] + 1 + j
                    c[:, table[r][dst // b], dst % b] = c[:, table[r][src // b], src % b]
        return dict(k_cache=kc, v_cache=vc, seq_len=None, free_blocks=None, free_count=None, status=None)
    H, G, D = case["kv_heads"], case["group"], case["dim"]
    par = _parents(case)
    see = torch.zeros(n, n, dtype=torch.bool)
    for j in range(n):
        x = j
        while x >= 0:
            see[j, x] = True
            x = par[x] if case["tree"] else x - 1
    hide = ~see.cuda().repeat_interleave(G, 0)
    out = torch.empty(R * n, H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(R * n, H * G, dtype=torch.float64, device="cuda")
    for r in range(R):
        ids = torch.tensor(table[r][: _up(L[r] + n, b)], device="cuda")
        for h in range(H):
            K = s["kc"][ids, :, h].reshape(-1, D)[: L[r] + n].double()
            V = s["vc"][ids, :, h].reshape(-1, D)[: L[r] + n].double()
            Q = s["q"][r * n:(r + 1) * n, h * G:(h + 1) * G].reshape(n * G, D).double()
            z = torch.einsum("id,xd->ix", Q, K) * s["scale"]
            z[:, L[r]:][hide] = -math.inf
            w = torch.logsumexp(z, 1)
            y = torch.einsum("ix,xd->id", torch.exp(z - w.unsqueeze(1)), V)
            out[r * n:(r + 1) * n, h * G:(h + 1) * G] = y.view(n, G, D)
            lse[r * n:(r + 1) * n, h * G:(h + 1) * G] = w.view(n, G)
    return dict(out=out, lse=lse)
