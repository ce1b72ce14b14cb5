"""The example's decoding, against one pass over each finished sequence with a cache of its own."""
import os
import sys

import pytest
import torch

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(sv):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import verify_step

    return verify_step


# Two passes of the same bf16 network sum in different orders.  Were each of some 20 roundings on a token's way to
# fall to the other side, that were sqrt(20) * 2^-8 = 0.02 of the states' size, 1.  The bound is six of that;
# unrelated logits differ by several units.
BOUND = 0.125


@pytest.mark.parametrize("R,prompt,length,K,every", [(8, 40, 96, 7, 5), (1, 2, 40, 1, 3), (3, 200, 60, 20, 4)])
def test_drafted_decoding_is_the_models_own(example, R, prompt, length, K, every):
    model, prompts, plain, drafted = example.main(R, prompt, length, K, every)
    assert all(len(row) == length for row in plain[1])
    more = 0
    for s, rows in (plain, drafted):
        steps = length if s is plain[0] else length // 5
        seq_len, table = s.seq_len.tolist(), s.table.cpu()
        for r, row in enumerate(rows):
            assert seq_len[r] == prompt - 1 + len(row)  # the root and what was accepted, step by step
            more += len(row) - steps
            fresh = example.Sessions(1, prompt + len(row))
            tokens = torch.cat([prompts[r], torch.tensor(row, device="cuda")])[:-1]
            n = tokens.numel()
            logits, step = example.forward(model, fresh, tokens,
                                           torch.full((1,), n, dtype=torch.int32, device="cuda"), None, n)
            assert step["status"].item() == 0
            own = logits[prompt - 1:].float()
            chosen = own.gather(1, torch.tensor(row, device="cuda")[:, None])[:, 0]
            assert (chosen >= own.max(1).values - 2 * BOUND).all(), (R, r)
            # what the cache holds for the committed tokens
            pos = torch.arange(seq_len[r], device="cuda")
            at = table[r].cuda().long()[pos // example.BLOCK], pos % example.BLOCK
            fat = fresh.table[0].long()[pos // example.BLOCK], pos % example.BLOCK
            for a, b in ((s.k, fresh.k), (s.v, fresh.v)):
                x, y = a[:, at[0], at[1]].float(), b[:, fat[0], fat[1]].float()
                assert ((x - y).abs() <= BOUND * (1 + y.abs())).all()
        # every block is owned once or free
        held = [b for r in range(R) for b in table[r, :-(-seq_len[r] // example.BLOCK)].tolist()]
        free = s.free[:s.free_count.item()].tolist()
        assert sorted(held + free) == list(range(s.k.shape[1]))
    assert more > 0  # drafts were accepted
