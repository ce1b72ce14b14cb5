"""Greedy speculative decoding over a paged cache, with every part of a step on the GPU.

A small decoder with random weights decodes a few sessions twice.  First a token a step.  Then with drafts of two
branches of K tokens a step: the tokens of the first decoding, with mistakes put in.  A step is

    step_tables     blocks, slots, positions and ancestor masks of the step's tokens
    rope_cache      per layer: rotary positions, keys and values into the cache
    tree_attention  per layer: the root and both branches over the session's cache
    verify_greedy   the drafts against the logits
    cache_commit    the accepted branch's keys and values kept, surplus blocks given back

Lengths, tables and the free list stay on the device; nothing of a step waits for the host.

    python examples/verify_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import serving_sampler_gb300 as sv  # noqa: E402

LAYERS, HEADS, KV_HEADS, HEAD_DIM, VOCAB, BLOCK = 3, 14, 2, 64, 512, 16


def make_model(seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = HEADS * HEAD_DIM

    def w(rows, cols):
        return (torch.randn(rows, cols, generator=g, device="cuda") * rows ** -0.5).to(dtype)

    layers = [dict(qkv=w(d, (HEADS + 2 * KV_HEADS) * HEAD_DIM), o=w(d, d), up=w(d, 2 * d), down=w(2 * d, d))
              for _ in range(LAYERS)]
    return dict(embed=w(VOCAB, d) * VOCAB ** 0.5, head=w(d, VOCAB), layers=layers,
                freqs=sv.rope_freqs(HEAD_DIM, 10000.0))


def norm(x):
    return torch.nn.functional.rms_norm(x, x.shape[-1:])


class Sessions:
    """The state of R sessions: committed tokens' keys and values, tables, lengths, free blocks."""

    def __init__(self, R, most, blocks=None, dtype=torch.bfloat16):
        self.R, per = R, -(-most // BLOCK)
        blocks = R * per if blocks is None else blocks
        shape = (LAYERS, blocks, BLOCK, KV_HEADS, HEAD_DIM)
        self.k, self.v = torch.empty(shape, dtype=dtype, device="cuda"), torch.empty(shape, dtype=dtype, device="cuda")
        self.table = torch.full((R, per), -1, dtype=torch.int32, device="cuda")
        self.seq_len = torch.zeros(R, dtype=torch.int32, device="cuda")
        self.free = torch.arange(blocks, dtype=torch.int32, device="cuda")
        self.free_count = torch.full((1,), blocks, dtype=torch.int32, device="cuda")


def forward(model, s, tokens, new_len, parent, most):
    """The step's tokens [T] laid out, cached and attended for: logits [T, VOCAB] and the step's tables."""
    T = tokens.numel()
    step = sv.step_tables(s.seq_len, new_len, s.table, s.free, s.free_count, BLOCK, T, parent=parent,
                          mask_words=(most + 31) // 32)
    x = model["embed"][tokens]
    for n, layer in enumerate(model["layers"]):
        qkv = (norm(x) @ layer["qkv"]).view(T, HEADS + 2 * KV_HEADS, HEAD_DIM)
        q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], 1)
        q = sv.rope_cache(q, k, v, step["position"], step["slot"], model["freqs"], s.k[n], s.v[n])
        a = sv.tree_attention(q, s.k[n], s.v[n], s.table, step["kv_len"], step["cu_tokens"], most,
                              mask=step.get("mask"))["out"]
        x = x + a.reshape(T, -1) @ layer["o"]
        x = x + torch.nn.functional.silu(norm(x) @ layer["up"]) @ layer["down"]
    return norm(x) @ model["head"], step


def prefill(model, s, prompts):
    """Prompts [R, n]: all but the last token are committed; the last is the first step's root."""
    R, n = prompts.shape
    new_len = torch.full((R,), n - 1, dtype=torch.int32, device="cuda")
    _, step = forward(model, s, prompts[:, :-1].reshape(-1), new_len, None, n - 1)
    s.seq_len, s.free_count = step["kv_len"], step["free_count"]
    return prompts[:, -1].to(torch.int32)


def parents(R, branches, k):
    """Parents of a root and `branches` chains of k drafts that follow it, for R sessions."""
    one = [-1] + [0 if i == 0 else b * k + i for b in range(branches) for i in range(k)]
    return torch.tensor(one, dtype=torch.int32).repeat(R).cuda()


def verify_step(model, s, root, draft):
    """One step for root [R] and draft [R, branches, k]: the tokens [R, k + 1] it yields (-1 behind the last one),
    and the next root."""
    R, branches, k = draft.shape
    n = 1 + branches * k
    tokens = torch.cat([root[:, None], draft.view(R, -1)], 1).reshape(-1).long()
    new_len = torch.full((R,), n, dtype=torch.int32, device="cuda")
    logits, step = forward(model, s, tokens, new_len, parents(R, branches, k), n)
    got = sv.verify_greedy(logits, R, k, branches, draft)
    kept = sv.cache_commit(s.k, s.v, s.table, s.seq_len, step["kv_len"], step["cu_tokens"], got["accept_len"], k,
                           s.free, step["free_count"], branch=got["branch"])
    s.seq_len, s.free_count = kept["seq_len"], kept["free_count"]
    return got, got["tokens"].gather(1, got["accept_len"][:, None].long())[:, 0]


def decode(model, prompts, steps, propose):
    """`steps` steps from `prompts`; propose(s) gives draft [R, branches, k] from the sessions' lengths.  Returns the
    sessions and, for each, the tokens behind its prompt."""
    R, n = prompts.shape
    s = Sessions(R, n + 16 * (steps + 1))
    root = prefill(model, s, prompts)
    yielded = []
    for _ in range(steps):
        got, root = verify_step(model, s, root, propose(s))
        yielded.append(got["tokens"])
    rows = torch.cat(yielded, 1).tolist()
    return s, [[t for t in row if t >= 0] for row in rows]


def main(R=8, prompt=40, length=96, K=7, every=5):
    """Both decodings: the model, the prompts, (sessions, tokens) a token a step, the same with drafts."""
    model = make_model()
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = torch.randint(VOCAB, (R, prompt), generator=g, device="cuda")
    none = torch.empty((R, 1, 0), dtype=torch.int32, device="cuda")
    plain = decode(model, prompts, length, lambda s: none)
    known = torch.nn.functional.pad(torch.tensor(plain[1], dtype=torch.int32), (0, K)).cuda()

    def propose(s):
        # a step's root is the last token so far, at position seq_len
        at = (s.seq_len - (prompt - 1)).long()[:, None] + torch.arange(K, device="cuda")
        right = known.gather(1, at.clamp(max=known.shape[1] - 1))
        wrong = (right + 1) % VOCAB
        first = torch.where(at % every == 0, wrong, right)          # the main branch errs now and then
        second = torch.where(at % every == every - 1, wrong, right)  # the other one elsewhere
        return torch.stack([first, second], 1).contiguous()

    return model, prompts, plain, decode(model, prompts, length // 5, propose)


if __name__ == "__main__":
    _, prompts, (_, plain), (_, drafted) = main()
    same = sum(a[:len(b)] == b[:len(a)] for a, b in zip(plain, drafted))
    print(f"{len(plain)} sessions: {len(plain[0])} tokens in {len(plain[0])} steps; with drafts "
          f"{sum(map(len, drafted)) / len(drafted):.1f} in {len(plain[0]) // 5}, the same ones in {same} sessions "
          f"(others part where two logits nearly tie)")
