"""Sessions from their first token to their last: prompts, forks, steps whose rows are penalised and masked and verified,
sessions that leave, a pool packed to its front, and forks again.  Every token that came out is checked against one pass
over its whole sequence with a cache of its own, under the same rules."""
import numpy as np
import pytest
import torch

from tests import pages_plain as plain
from tests.test_gpu_example import BOUND, example  # noqa: F401

pytestmark = pytest.mark.gpu

R, K, MOST = 6, 3, 160


def _forward(sv, e, model, s, tokens, new_len, most):
    """example.forward with a norm of every query and key head."""
    T = tokens.numel()
    step = sv.step_tables(s.seq_len, new_len, s.table, s.free, s.free_count, e.BLOCK, T)
    x = model["embed"][tokens]
    for n, layer in enumerate(model["layers"]):
        qkv = (e.norm(x) @ layer["qkv"]).view(T, e.HEADS + 2 * e.KV_HEADS, e.HEAD_DIM)
        q, k, v = qkv.split([e.HEADS, e.KV_HEADS, e.KV_HEADS], 1)
        q = sv.norm_rope_cache(q, k, v, step["position"], step["slot"], model["freqs"], s.k[n], s.v[n],
                               q_weight=model["q_weight"], k_weight=model["k_weight"])
        a = sv.tree_attention(q, s.k[n], s.v[n], s.table, step["kv_len"], step["cu_tokens"], most)["out"]
        x = x + a.reshape(T, -1) @ layer["o"]
        x = x + torch.nn.functional.silu(e.norm(x) @ layer["up"]) @ layer["down"]
    return e.norm(x) @ model["head"], step


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _owned(s, e):
    """Every block is free or held; a block that several rows hold is full of committed tokens in each."""
    seq = s.seq_len.tolist()
    held = [s.table[r, : -(-seq[r] // e.BLOCK)].tolist() for r in range(s.R)]
    free = s.free[: s.free_count.item()].tolist()
    ids = sorted(set(b for row in held for b in row))
    assert sorted(ids + free) == list(range(s.k.shape[1]))
    for r, row in enumerate(held):
        for i, b in enumerate(row):
            others = [q for q in range(s.R) if q != r and b in held[q]]
            assert not others or (i + 1) * e.BLOCK <= seq[r]


def test_sessions(sv, example):  # noqa: F811
    e, rng = example, np.random.default_rng(3)
    model = e.make_model()
    g = torch.Generator(device="cuda").manual_seed(9)
    for name in ("q_weight", "k_weight"):
        model[name] = (1 + 0.3 * torch.randn(e.HEAD_DIM, generator=g, device="cuda")).bfloat16()
    V, n = e.VOCAB, 1 + K
    s = e.Sessions(R, MOST)
    prompts = [rng.integers(0, V, m).tolist() for m in (37, 49)]  # 36 and 48 committed tokens: a part and full blocks
    texts = [list(prompts[0]), list(prompts[1]), [], [], [], []]
    told = [len(t) for t in texts]  # of each text, the prompt
    cached = [p[:-1] for p in prompts]
    _, step = _forward(sv, e, model, s, torch.tensor(sum(cached, []), device="cuda"),
                       _ints([len(c) for c in cached] + [0] * 4), 48)
    assert not step["status"].any()
    s.seq_len, s.free_count = step["kv_len"] + 0, step["free_count"]

    rules = dict(repetition=torch.linspace(0.9, 1.5, R, device="cuda"), presence=torch.linspace(0, 0.6, R, device="cuda"),
                 frequency=torch.linspace(0.3, 0, R, device="cuda"))
    bias = (_ints([0, 2, 2, 3, 3, 4, 4]), _ints([5, 6, 7, 8]), torch.tensor([1.0, -np.inf, 3.0, -2.0], device="cuda"))
    said = []  # (text before the token, its prompt, row, mask, token)

    def fork(source):
        got = sv.cache_fork(s.k, s.v, s.table, s.seq_len, _ints(source), s.free, s.free_count)
        assert not got["status"].any()
        s.seq_len, s.free_count = got["seq_len"], got["free_count"]
        for r, q in enumerate(source):
            if q >= 0:
                texts[r], told[r] = list(texts[q]), told[q]
        _owned(s, e)

    def steps(count):
        accepted = 0
        for _ in range(count):
            allowed = rng.random((R * n, V)) < 0.5
            picks = rng.integers(0, V, (R * n, 3))
            allowed[::2] = False
            allowed[np.arange(R * n)[:, None], picks] = True  # a bracket, or nearly any text
            bits = np.packbits(allowed, axis=1, bitorder="little").view(np.int32)
            draft = _ints(picks.reshape(R, n, 3)[:, :K, 0].reshape(R, 1, K).tolist())
            roots = torch.tensor([t[-1] for t in texts], device="cuda")
            tokens = torch.cat([roots[:, None], draft[:, 0].long()], 1).reshape(-1)
            logits, step = _forward(sv, e, model, s, tokens, _ints([n] * R), n)
            width = max(map(len, texts)) + 3
            history = _ints([t + [-1] * (width - len(t)) for t in texts])
            got = sv.adjust_logits(logits, R, K, 1, draft, history=history, history_len=_ints([len(t) for t in texts]),
                                   prompt_len=_ints(told), bias=bias, mask=torch.from_numpy(bits).cuda(), **rules,
                                   out=dict(logits=logits, status=torch.empty(R, dtype=torch.int32, device="cuda")))
            assert not got["status"].any() and not step["status"].any()
            got = sv.verify_greedy(logits, R, K, 1, draft)
            kept = sv.cache_commit(s.k, s.v, s.table, s.seq_len, step["kv_len"], step["cu_tokens"], got["accept_len"], K,
                                   s.free, step["free_count"])
            s.seq_len, s.free_count = kept["seq_len"], kept["free_count"]
            for r, (m, row) in enumerate(zip(got["accept_len"].tolist(), got["tokens"].tolist())):
                accepted += m
                for j, token in enumerate(row[: m + 1]):
                    said.append((list(texts[r]), told[r], r, allowed[r * n + j], token))
                    texts[r].append(token)
        _owned(s, e)
        return accepted

    fork([-1, -1, 0, 0, 1, 0])
    accepted = steps(8)
    left = s.free_count.item()
    got = sv.cache_free(s.table, s.seq_len, _ints([1, 0, 0, 0, 1, 0]), s.free, s.free_count, e.BLOCK)
    s.seq_len, s.free_count = got["seq_len"], got["free_count"]
    assert s.seq_len.tolist()[0] == 0 and s.free_count.item() > left
    texts[0], texts[4] = [], []
    _owned(s, e)
    got = sv.cache_compact(s.k, s.v, s.table, s.seq_len)
    s.table, s.free, s.free_count = got["block_table"], got["free_blocks"], got["free_count"]
    assert s.table.max().item() == s.k.shape[1] - s.free_count.item() - 1  # the front of the pool
    _owned(s, e)
    fork([3, -1, -1, -1, 1, -1])
    accepted += steps(8)
    assert accepted > 0
    lengths = s.seq_len.tolist()
    assert lengths == [len(t) - 1 for t in texts]

    for text, prompt, r, allowed, token in said:
        fresh = e.Sessions(1, MOST)
        logits, _ = _forward(sv, e, model, fresh, torch.tensor(text, device="cuda"), _ints([len(text)]), len(text))
        one = {name: [float(x[r])] for name, x in rules.items()}
        b0, b1 = int(bias[0][r]), int(bias[0][r + 1])
        mask = np.packbits(allowed[None], axis=1, bitorder="little").view(np.int32)
        z, _, _ = plain.adjust(logits[-1:].double().cpu().numpy(), 1, 0, 1, None, np.array([text]), [len(text)], [prompt],
                               bias=(np.array([0, b1 - b0]), bias[1][b0:b1].tolist(), bias[2][b0:b1].tolist()), mask=mask, **one)
        # both sides of the comparison are off by the example's bound times the largest penalty's factor, 1.5
        assert z[0, token] >= z.max() - 2 * 1.5 * BOUND, (r, len(text), z[0, token], z.max())
