"""Cases for the operators at the two ends of a verify step: logits on their way into verification, queries and keys on
their way into the paged cache, and the pages that sessions begin and end with.

  adjust   adjust_logits: penalties for repeated tokens, biases and grammar masks on the rows of a verify step
  norm     norm_rope_cache: an RMS norm of every query and key head, rotary positions, k and v into their cache slots
  fork     cache_fork: sessions branched into several that share their full blocks, the last block copied
  free     cache_free: the blocks of leaving sessions that no staying one holds, pushed on the free stack
  compact  cache_compact: the held blocks moved to the front of the pool, tables and free stack rewritten

A verify step's request has 1 + branches * k rows: the first one, then the rows behind each draft of each branch.  `run`
computes an operator in elementary torch operations, or calls the package's own entry points where `own` is true.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _adjust(name, R, branches, k, V, lo, hi, biases, masks, dtype):
    """lo .. hi: tokens of a session so far; biases: entries a request; masks: of every `masks` rows one has none (0: no masks)."""
    return dict(name=name, op="adjust", R=R, branches=branches, k=k, V=V, lo=lo, hi=hi, biases=biases, masks=masks,
                dtype=dtype)


def _norm(name, T, hi, heads, kv_heads, dim, rot, interleaved, weights, block, dtype):
    return dict(name=name, op="norm", T=T, hi=hi, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                interleaved=interleaved, weights=weights, block=block, dtype=dtype)


def _fork(name, R, each, lo, hi, layers, kv_heads, dim, block, dtype):
    """R sessions, each branched into `each` more."""
    return dict(name=name, op="fork", R=R, each=each, lo=lo, hi=hi, layers=layers, kv_heads=kv_heads, dim=dim,
                block=block, dtype=dtype)


def _free(name, R, lo, hi, leave, block):
    """Of R sessions, every second a fork of the one before, one in `leave` leaves."""
    return dict(name=name, op="free", R=R, lo=lo, hi=hi, leave=leave, block=block)


def _compact(name, R, lo, hi, layers, kv_heads, dim, block, dtype):
    """R sessions, every second a fork of the one before, over a pool of twice the blocks they hold."""
    return dict(name=name, op="compact", R=R, lo=lo, hi=hi, layers=layers, kv_heads=kv_heads, dim=dim, block=block,
                dtype=dtype)


def listed():
    return [
        # one session decoding a token a step with penalties: a single row of the large vocabulary
        _adjust("adjust-1x1", 1, 1, 0, 151936, 777, 777, 0, 0, "bf16"),
        # a serving batch verifying chains of 8 drafts, a grammar on two rows of three, a few banned and favoured tokens
        _adjust("adjust-64x9", 64, 1, 8, 151936, 500, 8000, 16, 3, "bf16"),
        # 17 requests with two branches of 16 drafts, fp32 rows of an odd vocabulary, every row masked by the grammar
        _adjust("adjust-17x33", 17, 2, 16, 32003, 0, 3000, 100, 1, "fp32"),
        # a single token in one layer: the plain decode step
        _norm("norm-1", 1, 1000, 32, 8, 128, 128, False, "bf16", 16, "bf16"),
        # 64 listening sessions of 65 tokens, half of each head rotated, pairs side by side, fp32 weights
        _norm("norm-4160", 4160, 4000, 28, 4, 128, 64, True, "fp32", 64, "bf16"),
        # long draft chains, a head size that is no power of two
        _norm("norm-15420", 15420, 9000, 32, 8, 96, 96, False, "fp16", 32, "fp16"),
        # one session branched into seven candidate replies, a few layers' cache
        _fork("fork-1x7", 1, 7, 1000, 1000, 4, 8, 128, 16, "bf16"),
        # listening sessions that each get a second reply, the caches of 16 layers
        _fork("fork-64x1", 64, 1, 100, 1000, 16, 4, 128, 64, "bf16"),
        # a small batch, two sessions of which leave
        _free("free-8", 8, 100, 1000, 4, 16),
        # the largest batch of the throughput sweep, every other session leaves
        _free("free-1024", 1024, 100, 6000, 2, 16),
        # a small pool of a few layers
        _compact("compact-4", 4, 50, 90, 4, 8, 128, 16, "bf16"),
        # listening sessions' caches of 16 layers after half of the pool was given back
        _compact("compact-64", 64, 100, 1500, 16, 4, 128, 64, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adjust", "adjust", "adjust", "norm", "norm", "fork", "free", "compact"])
    block = rng.choice([8, 16, 16, 24, 32, 48, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "adjust":
        V = rng.choice([151936, 32000, 4096, _log(rng, 100, 200000)])
        branches = rng.choice([1, 1, 2, 3, 8])
        k = rng.choice([0, _log(rng, 1, 32), _log(rng, 1, 32)]) if branches == 1 else _log(rng, 1, 32)
        R = _log(rng, 1, 256)
        dtype = rng.choice(["bf16", "fp32"])
        least = 0 if branches == 1 else 1
        while R * (1 + branches * k) * V > 64 * 8 * 151936 // (1 if dtype == "bf16" else 2):
            R, k = (R - 1 - R // 8, k) if R > 8 else (R, k - 1) if k > least else (max(1, R - 1), k)
        hi = _log(rng, 1, 8000)
        return _drop(_adjust("", R, branches, k, V, rng.randint(0, hi), hi, rng.choice([0, 0, 1, 16, _log(rng, 1, 300)]),
                             rng.choice([0, 1, 2, 3, 5]), dtype))
    if op == "free":
        hi, R = _log(rng, 2, 5000), _log(rng, 2, 1024)
        block = max(block, 16)
        return _drop(_free("", R, rng.randint(0, hi), hi, rng.randint(2, 8), block))
    dim = rng.choice([64, 80, 96, 128, 128, rng.randrange(8, 129, 8)])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
    if op == "norm":
        T, group = _log(rng, 1, 15420), rng.choice([1, 2, 4, 5, 7, 8])
        while T * kv_heads * (group + 2) * dim > 15420 * 48 * 96:
            T = max(1, T - 1 - T // 8)
        rot = min(dim, rng.choice([dim, dim, dim // 2, max(2, dim // 4 * 2)]) // 2 * 2)
        return _drop(_norm("", T, _log(rng, 2, 131000), kv_heads * group, kv_heads, dim, rot, rng.random() < 0.5,
                           rng.choice([dtype, "fp32", "none"]), block, dtype))
    layers = _log(rng, 1, 16)
    if op == "fork":
        R, each, hi = _log(rng, 1, 64), rng.choice([1, 1, 2, 3, 7]), _log(rng, 2, 1000)
        # whole caches come back: both their size and what is copied stay within the largest listed case's
        while (R * (hi + block) + R * each * block) * layers * kv_heads * dim > 64 * (1064 + 64) * 16 * 4 * 128 \
                or R * each * block * layers * kv_heads * dim > 64 * 32 * 16 * 4 * 128:
            R, layers = max(1, R // 2), max(1, layers - 1)
            hi = max(2, hi - hi // 8)
        return _drop(_fork("", R, each, rng.randint(0, hi), hi, layers, kv_heads, dim, block, dtype))
    R, hi = _log(rng, 1, 64), _log(rng, 2, 1500)
    while R * (hi + block) * layers * kv_heads * dim > 64 * 1564 * 16 * 4 * 128 // 2:
        R, layers = max(1, R // 2), max(1, layers - 1)
    return _drop(_compact("", R, rng.randint(0, hi), hi, layers, kv_heads, dim, block, dtype))


def _drop(case):
    case.pop("name")
    return case


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _lengths(case):
    """Tokens of each session: the ends of the range and values between, a part of the case."""
    rng = random.Random(case["R"] * 1000003 + case["lo"] * 1009 + case["hi"])
    got = [case["hi"], case["lo"]] + [rng.randint(case["lo"], case["hi"]) for _ in range(case["R"])]
    return got[: case["R"]]


def _rows(case):
    return 1 + case["branches"] * case["k"]


def _up(a, b):
    return -(-a // b)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _shared(case):
    """Full blocks that each session shares with the one before: every second one is a fork of its neighbour, taken
    when that had half of the shorter one's tokens."""
    L = _lengths(case)
    return [min(L[r], L[r - 1]) // 2 // case["block"] if r % 2 else 0 for r in range(case["R"])]


def _pool(case, g, blocks, L, shared):
    """A block table over a shuffled pool and the stack of the blocks that no session holds."""
    b, R = case["block"], len(L)
    held = [_up(x, b) for x in L]
    mine = [held[r] - shared[r] for r in range(R)]
    most = max(max(held), 1) + 1
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((R, most), -1, dtype=torch.int32, device="cuda")
    cols = torch.arange(most, device="cuda").view(1, -1)
    first = torch.tensor(shared, device="cuda").view(-1, 1)
    table[(cols >= first) & (cols < torch.tensor(held, device="cuda").view(-1, 1))] = order[: sum(mine)]
    before = table[torch.arange(R, device="cuda") - 1]
    table = torch.where(cols < first, before, table)
    free = torch.full((blocks,), -1, dtype=torch.int32, device="cuda")
    left = blocks - sum(mine)
    free[:left] = order[sum(mine):]
    return dict(table=table.contiguous(), blocks=blocks, free=free, free_count=_ints([left]), seq_len=_ints(L))


def _freqs(case):
    """Turns per position of each pair as 64-bit fractions: 2^64 inv_freq / (2 pi)."""
    half = case["rot"] // 2
    out = []
    for i in range(half):
        x = int(round(10000.0 ** (-i / half) / (2 * math.pi) * 2.0 ** 64))
        out.append(x - 2 ** 64 if x >= 2 ** 63 else x)
    return torch.tensor(out, dtype=torch.int64, device="cuda")


def _masked_rows(case):
    """The mask of each row: of every `masks` rows the last has none (all have one where masks is 1)."""
    n, m = case["R"] * _rows(case), case["masks"]
    return [-1 if m > 1 and i % m == m - 1 else i for i in range(n)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = dict(case=case)
    if op == "adjust":
        R, V, n, L = case["R"], case["V"], _rows(case), _lengths(case)
        width = max(L) + 8
        # texts repeat themselves: most tokens come from a few hundred of the vocabulary, the rest from all of it
        few = torch.randint(0, V, (R, 400), generator=g, device="cuda", dtype=torch.int32)

        def tokens(*shape):
            pick = torch.randint(0, 400, shape, generator=g, device="cuda")
            rare = torch.randint(0, V, shape, generator=g, device="cuda", dtype=torch.int32)
            often = torch.rand(shape, generator=g, device="cuda") < 0.7
            return torch.where(often, few.gather(1, pick.view(R, -1)).view(shape), rare)

        s.update(R=R, k=case["k"], branches=case["branches"],
                 logits=(torch.randn(R * n, V, generator=g, device="cuda") * 3).to(DTYPES[case["dtype"]]),
                 draft=tokens(R, case["branches"], case["k"]), history=tokens(R, width), history_len=_ints(L),
                 prompt_len=_ints([x // 3 for x in L]),
                 repetition=1.0 + 0.3 * torch.rand(R, generator=g, device="cuda"),
                 presence=0.5 * torch.rand(R, generator=g, device="cuda"),
                 frequency=0.2 * torch.rand(R, generator=g, device="cuda"), bias=None, mask=None, mask_row=None)
        if case["biases"]:
            m = min(case["biases"], V)  # each id once a request: a stride that meets no id twice
            start = torch.randint(0, V, (R, 1), generator=g, device="cuda")
            ids = (start + torch.arange(m, device="cuda").view(1, m) * (V // m)) % V
            value = torch.randn(R, m, generator=g, device="cuda") * 2
            value = torch.where(torch.rand(R, m, generator=g, device="cuda") < 0.2, -math.inf, value)  # banned
            s["bias"] = (_ints(range(0, R * m + 1, m)), ids.to(torch.int32).reshape(-1), value.reshape(-1))
        if case["masks"]:
            words = _up(V, 32)
            # a grammar allows long stretches (any text) or next to nothing (a bracket): by stretches of 256 tokens
            dense = torch.rand(R * n, _up(words, 8), 1, generator=g, device="cuda") < torch.rand(R * n, 1, 1, generator=g, device="cuda")
            bits = torch.randint(-2 ** 31, 2 ** 31, (R * n, _up(words, 8), 8), generator=g, device="cuda")
            rare = bits & bits.roll(1, 1) & bits.roll(2, 1) & bits.roll(3, 1)
            s["mask"] = torch.where(dense, -1, rare).view(R * n, -1)[:, :words].to(torch.int32).contiguous()
            s["mask_row"] = _ints(_masked_rows(case))
        return s
    if op == "norm":
        T, Hq, H, D, dt = case["T"], case["heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
        # one projection's output, whose heads differ in size by a few times; q, k and v are views of it
        size = torch.exp(torch.randn(1, Hq + 2 * H, 1, generator=g, device="cuda"))
        qkv = (torch.randn(T, Hq + 2 * H, D, generator=g, device="cuda") * size).to(dt)
        blocks = _up(T, case["block"]) + 5
        w = case["weights"]
        q_weight, k_weight = (None if w == "none" else (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(DTYPES[w])
                              for _ in range(2))
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + H], v=qkv[:, Hq + H:], q_weight=q_weight, k_weight=k_weight, eps=1e-6,
                 slot=torch.randperm(blocks * case["block"], generator=g, device="cuda")[:T].contiguous(),
                 position=torch.randint(0, case["hi"] + 1, (T,), generator=g, device="cuda", dtype=torch.int32),
                 freqs=_freqs(case), interleaved=case["interleaved"],
                 kc=torch.zeros(blocks, case["block"], H, D, dtype=dt, device="cuda"),
                 vc=torch.zeros(blocks, case["block"], H, D, dtype=dt, device="cuda"))
        return s
    b, L = case["block"], _lengths(case)
    R = case["R"]
    if op == "fork":
        each = case["each"]
        L = L + [0] * (R * each)
        s.update(_pool(case, g, sum(_up(x, b) for x in L) + R * each + 3, L, [0] * len(L)))
        s.update(source=_ints([-1] * R + [i // each for i in range(R * each)]))
    else:
        shared = _shared(case)
        mine = sum(_up(x, b) for x in L) - sum(shared)
        s.update(_pool(case, g, 2 * mine + 3, L, shared))
        if op == "free":  # seeded: who leaves is not known before
            leave = torch.randint(0, case["leave"], (R,), generator=g, device="cuda") == 0
            s.update(leave=leave.to(torch.int32), block=b)
            return s
    dt = DTYPES[case["dtype"]]
    shape = (case["layers"], s["blocks"], b, case["kv_heads"], case["dim"])
    s.update(kc=torch.randn(shape, generator=g, device="cuda", dtype=dt),
             vc=torch.randn(shape, generator=g, device="cuda", dtype=dt))
    return s


# ---------------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------------
def _plain_adjust(s):
    z = s["logits"].float()
    rows, V = z.shape
    R, k, branches = s["R"], s["k"], s["branches"]
    n = rows // R
    h = s["history"].long()
    at = torch.arange(h.shape[1], device="cuda").view(1, -1)
    there = at < s["history_len"].view(R, 1)
    out = there & (at >= s["prompt_len"].view(R, 1))
    counts = torch.zeros(R, V, device="cuda").scatter_add_(1, h, out.float())
    seen = torch.zeros(R, V, device="cuda").scatter_add_(1, h, there.float())
    counts, seen = counts.repeat_interleave(n, 0), seen.repeat_interleave(n, 0)
    if k:
        # the drafts before each row: row 1 + b k + i has the first i + 1 of branch b
        i = torch.arange(k, device="cuda")
        path = (i.view(1, k) <= i.view(k, 1)).float()  # [row behind draft i, draft]
        path = torch.cat([torch.zeros(1, k, device="cuda"), path.repeat(branches, 1)]).repeat(R, 1)
        one = s["draft"].long()
        ids = torch.cat([one[:, :1], one.repeat_interleave(k, 1)], 1).view(rows, k)
        counts.scatter_add_(1, ids, path)
        seen.scatter_add_(1, ids, path)
    rep, pres, freq = (s[x].repeat_interleave(n).view(rows, 1) for x in ("repetition", "presence", "frequency"))
    z = torch.where(seen > 0, torch.where(z > 0, z / rep, z * rep), z)
    z = torch.where(counts > 0, z - (pres + freq * counts), z)
    if s["bias"] is not None:
        start, ids, value = s["bias"]
        bias = torch.zeros(R, V, device="cuda").scatter_(1, ids.long().view(R, -1), value.view(R, -1))
        z = z + bias.repeat_interleave(n, 0)
    if s["mask"] is not None:
        x = torch.arange(V, device="cuda")
        masked = (s["mask"][s["mask_row"].long().clamp(min=0)][:, x // 32] >> (x % 32)) & 1 == 0
        z = z.masked_fill(masked & (s["mask_row"] >= 0).view(rows, 1), -math.inf)
    return dict(logits=z.to(s["logits"].dtype), status=torch.zeros(R, dtype=torch.int32, device="cuda"))


def _plain_rotate(x, c, sn, interleaved):
    rot = 2 * c.shape[-1]
    a, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        u, w = a[..., 0::2], a[..., 1::2]
        y = torch.stack([u * c - w * sn, u * sn + w * c], -1).flatten(-2)
    else:
        u, w = a[..., : rot // 2], a[..., rot // 2:]
        y = torch.cat([u * c - w * sn, u * sn + w * c], -1)
    return torch.cat([y, rest], -1)


def _plain_norm(s):
    phase = s["position"].long().view(-1, 1) * s["freqs"].view(1, -1)  # wraps: whole turns drop out
    angle = (phase >> 32).float() * (2 * math.pi / 2.0 ** 32)
    c, sn = torch.cos(angle).unsqueeze(1), torch.sin(angle).unsqueeze(1)

    def one(x, weight):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"])
        y = y if weight is None else y * weight.float()
        return _plain_rotate(y, c, sn, s["interleaved"]).to(x.dtype)

    s["kc"].view(-1, *s["kc"].shape[2:])[s["slot"]] = one(s["k"], s["k_weight"])
    s["vc"].view(-1, *s["vc"].shape[2:])[s["slot"]] = s["v"]
    return dict(q=one(s["q"], s["q_weight"]), k_cache=s["kc"], v_cache=s["vc"])


def _plain_fork(s):
    b = s["kc"].shape[2]
    table, L, src = s["table"].long(), s["seq_len"].long(), s["source"].long()
    R, most = table.shape
    forks = src >= 0
    src = src.clamp(min=0)
    new = torch.where(forks, L[src], L)
    need = (forks & (new % b > 0)).long()
    pre = need.cumsum(0) - need
    count = s["free_count"].long()
    fits = pre + need <= count
    fresh = s["free"][(count - 1 - pre).clamp(min=0)].long()
    cols = torch.arange(most, device="cuda").view(1, -1)
    takes = (forks & fits).view(R, 1)
    last = torch.where(need > 0, new // b, most).view(R, 1)
    rows = torch.where(takes & (cols < ((new + b - 1) // b).view(R, 1)), table[src], table)
    rows = torch.where(takes & (cols == last), fresh.view(R, 1), rows)
    j = torch.arange(b, device="cuda").view(1, b)
    move = takes & (need > 0).view(R, 1) & (j < (new % b).view(R, 1))
    old = table[src].gather(1, (new // b).clamp(max=most - 1).view(R, 1))
    at_from, at_to = (old * b + j)[move], (fresh.view(R, 1) * b + j)[move]
    for c in (s["kc"], s["vc"]):
        flat = c.view(c.shape[0], -1, *c.shape[3:])
        flat[:, at_to] = flat[:, at_from]
    s["table"].copy_(rows)
    return dict(k_cache=s["kc"], v_cache=s["vc"], block_table=s["table"], seq_len=torch.where(fits, new, L).int(),
                free_count=(count - (need * fits).sum()).int(), status=torch.where(fits, 0, 256).int())


def _held(table, seq_len, block):
    cols = torch.arange(table.shape[1], device="cuda").view(1, -1)
    return cols < ((seq_len.long() + block - 1) // block).view(-1, 1)


def _marks(ids, inside, blocks):
    """Which blocks are among the ids for which `inside` is true."""
    got = torch.zeros(blocks + 1, dtype=torch.bool, device="cuda")
    got.scatter_(0, torch.where(inside, ids.long(), blocks).view(-1), True)
    return got[:blocks]


def _plain_free(s):
    N, count, leave = s["blocks"], s["free_count"].long(), s["leave"] > 0
    held = _held(s["table"], s["seq_len"], s["block"])
    stay = _marks(s["table"], held & ~leave.view(-1, 1), N)
    gone = _marks(s["table"], held & leave.view(-1, 1), N)
    i = torch.arange(N, device="cuda")
    freed = gone & ~stay & ~_marks(s["free"], i < count, N)
    to = torch.where(freed, count + freed.long().cumsum(0) - 1, N)
    s["free"].copy_(torch.cat([s["free"], s["free"][:1]]).scatter_(0, to, i.int())[:N])
    return dict(seq_len=torch.where(leave, 0, s["seq_len"]), free_blocks=s["free"],
                free_count=(count + freed.sum()).int(), status=torch.zeros_like(s["seq_len"]))


def _plain_compact(s):
    N, b = s["blocks"], s["kc"].shape[2]
    held = _held(s["table"], s["seq_len"], b)
    used = _marks(s["table"], held, N)
    U = used.sum()
    i = torch.arange(N, device="cuda")
    high, gap = used & (i >= U), ~used & (i < U)
    gaps = torch.zeros(N + 1, dtype=torch.int64, device="cuda")
    gaps.scatter_(0, torch.where(gap, gap.long().cumsum(0) - 1, N), i)
    to = torch.where(high, gaps[(high.long().cumsum(0) - 1).clamp(min=0)], i)
    for c in (s["kc"], s["vc"]):
        c[:, to[high]] = c[:, high]
    table = torch.where(held, to[s["table"].long().clamp(min=0)], -1).int()
    return dict(k_cache=s["kc"], v_cache=s["vc"], block_table=table,
                free_blocks=torch.where(i < N - U, N - 1 - i, -1).int(), free_count=(N - U).view(1).int(),
                status=torch.zeros_like(s["seq_len"]))


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"adjust": _plain_adjust, "norm": _plain_norm, "fork": _plain_fork, "free": _plain_free,
                "compact": _plain_compact}[op](state)
    import serving_sampler_gb300 as sv

    s = state
    if op == "adjust":
        return sv.adjust_logits(s["logits"], s["R"], s["k"], s["branches"], s["draft"], history=s["history"],
                                history_len=s["history_len"], prompt_len=s["prompt_len"], repetition=s["repetition"],
                                presence=s["presence"], frequency=s["frequency"], bias=s["bias"], mask=s["mask"],
                                mask_row=s["mask_row"])
    if op == "norm":
        q = sv.norm_rope_cache(s["q"], s["k"], s["v"], s["position"], s["slot"], s["freqs"], s["kc"], s["vc"],
                               q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                               interleaved=s["interleaved"])
        return dict(q=q, k_cache=s["kc"], v_cache=s["vc"])
    if op == "fork":
        got = sv.cache_fork(s["kc"], s["vc"], s["table"], s["seq_len"], s["source"], s["free"], s["free_count"])
        return dict(got, k_cache=s["kc"], v_cache=s["vc"], block_table=s["table"])
    if op == "free":
        got = sv.cache_free(s["table"], s["seq_len"], s["leave"], s["free"], s["free_count"], s["block"])
        return dict(got, free_blocks=s["free"])
    if "workspace" not in s:  # kept by the program
        s["workspace"] = torch.empty(sv.cache_compact_workspace(s["blocks"]), dtype=torch.uint8, device="cuda")
    got = sv.cache_compact(s["kc"], s["vc"], s["table"], s["seq_len"], workspace=s["workspace"])
    return dict(got, k_cache=s["kc"], v_cache=s["vc"])


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    op, R = case["op"], case.get("R", 0)
    if op == "adjust":
        n, V, L = _rows(case), case["V"], _lengths(case)
        size = 2 if case["dtype"] == "bf16" else 4
        masked = sum(i >= 0 for i in _masked_rows(case)) if case["masks"] else 0
        small = 4 * sum(L) + 4 * R * (n - 1) + 24 * R + (8 * min(case["biases"], V) + 4) * R
        return dict(bytes=2 * size * R * n * V + masked * _up(V, 8) + small, flops=float(R * n * V))
    if op == "norm":
        T, rows, D = case["T"], case["heads"] + 2 * case["kv_heads"], case["dim"]
        turned = T * (case["heads"] + case["kv_heads"])
        return dict(bytes=2 * 2 * T * rows * D + 12 * T + 4 * case["rot"] + 8 * D,
                    flops=4.0 * turned * D + 3.0 * turned * case["rot"] + 40.0 * T * case["rot"] / 2)
    b, L = case["block"], _lengths(case)
    if op == "fork":
        tails = case["each"] * sum(x % b for x in L)
        entries = case["each"] * sum(_up(x, b) for x in L)
        return dict(bytes=2 * 2 * 2 * tails * case["layers"] * case["kv_heads"] * case["dim"] + 8 * entries
                    + 16 * R * (1 + case["each"]), flops=float(R * (1 + case["each"])))
    shared = _shared(case)
    entries, mine = sum(_up(x, b) for x in L), sum(_up(x, b) for x in L) - sum(shared)
    if op == "free":  # one in `leave` leaves on average
        return dict(bytes=4 * entries + 4 * mine / case["leave"] + 16 * R, flops=float(entries))
    # about half of the held blocks of a shuffled pool twice as large lie above them
    moved = mine / 2
    return dict(bytes=2 * 2 * 2 * moved * b * case["layers"] * case["kv_heads"] * case["dim"] + 8 * entries + 8 * mine,
                flops=float(entries))


# ---------------------------------------------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    if op == "free":
        return None  # whole numbers alone
    s = prepare(case, seed)
    if op == "adjust":
        R, n, k, V = case["R"], _rows(case), case["k"], case["V"]
        L = _lengths(case)
        got = s["logits"].double()
        bits = torch.arange(32, device="cuda")
        for r in range(R):
            tokens = s["history"][r, : L[r]].long()
            before = torch.bincount(tokens, minlength=V)
            said = torch.bincount(tokens[L[r] // 3:], minlength=V)
            rep, pres, freq = (float(s[x][r]) for x in ("repetition", "presence", "frequency"))
            for j in range(n):
                b, i = divmod(j - 1, k) if j else (0, -1)
                way = torch.bincount(s["draft"][r, b, : i + 1].long(), minlength=V)
                z, count = got[r * n + j], said + way
                up = z > 0
                z[up & (before + way > 0)] /= rep
                z[~up & (before + way > 0)] *= rep
                z -= torch.where(count > 0, pres + freq * count.double(), 0.0)
                if s["bias"] is not None:
                    m = s["bias"][1].numel() // R
                    z.index_add_(0, s["bias"][1][r * m:(r + 1) * m].long(), s["bias"][2][r * m:(r + 1) * m].double())
        if case["masks"]:
            for i, m in enumerate(_masked_rows(case)):
                if m >= 0:
                    ok = ((s["mask"][m].view(-1, 1) >> bits) & 1).view(-1)[:V] > 0
                    got[i, ~ok] = -math.inf
        return dict(logits=got, status=None)
    if op == "norm":
        pos = s["position"].tolist()
        turns = [int(x) % 2 ** 64 for x in s["freqs"].tolist()]
        half = case["rot"] // 2
        kinds = sorted(set(pos))
        ang = torch.tensor([[(p * f % 2 ** 64) / 2.0 ** 64 for f in turns] for p in kinds], dtype=torch.float64)
        row = {p: i for i, p in enumerate(kinds)}
        ang = (ang * (2 * math.pi)).view(len(kinds), half).cuda()[torch.tensor([row[p] for p in pos], device="cuda")]
        first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        done = []
        for x, weight in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            y = x.double()
            y = y / (torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / case["dim"] + s["eps"]).sqrt()
            if weight is not None:
                y = y * weight.double()
            u, w = y[:, :, first].clone(), y[:, :, second].clone()
            turn = torch.polar(torch.ones_like(ang), ang).unsqueeze(1) * torch.complex(u, w)
            y[:, :, first], y[:, :, second] = turn.real, turn.imag
            done.append(y)
        kc, vc = s["kc"].double(), s["vc"].double()
        at = (s["slot"] // case["block"], s["slot"] % case["block"])
        kc[at], vc[at] = done[1], s["v"].double()
        return dict(q=done[0], k_cache=kc, v_cache=vc)
    L, b = _lengths(case), case["block"]
    kc, vc = s["kc"].double(), s["vc"].double()
    table = s["table"].tolist()
    if op == "fork":
        free, top = s["free"].tolist(), int(s["free_count"])
        for i in range(case["R"] * case["each"]):
            r = i // case["each"]
            if L[r] % b:
                top -= 1
                for c in (kc, vc):
                    c[:, free[top], : L[r] % b] = c[:, table[r][L[r] // b], : L[r] % b]
        return dict(k_cache=kc, v_cache=vc, block_table=None, seq_len=None, free_count=None, status=None)
    used = sorted({x for r in range(case["R"]) for x in table[r][: _up(L[r], b)]})
    gaps = sorted(set(range(len(used))) - set(used))
    high = [x for x in used if x >= len(used)]
    for c in (kc, vc):
        for x, y in zip(high, gaps):
            c[:, y] = c[:, x]
    return dict(k_cache=kc, v_cache=vc, block_table=None, free_blocks=None, free_count=None, status=None)
