"""Calls whose dynamic shared memory lies just below what a kernel may have without asking for more, in a process of their
own: once a kernel was allowed more, every later call of it has it."""
import subprocess
import sys

import pytest

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

HEAD = """
import torch
import serving_sampler_gb300 as sv

ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")


def adjust(R, k, branches, V, width, in_place, biases=0):
    # presence 1 for the history's only token in every row, drafts of another one
    rows = 1 + branches * k
    z = torch.zeros((R * rows, V), dtype=torch.bfloat16, device="cuda")
    history = torch.zeros((R, width), dtype=torch.int32, device="cuda")
    history[:, 0] = torch.arange(R, device="cuda") % (V - 1)
    draft = torch.full((R, branches, k), V - 1, dtype=torch.int32, device="cuda")
    bias = None
    if biases:
        bias = (torch.arange(R + 1, dtype=torch.int32, device="cuda") * biases,
                (torch.arange(R * biases, device="cuda") % V).to(torch.int32), torch.zeros(R * biases, device="cuda"))
    status = ints([-1] * R)
    out = dict(logits=z if in_place else torch.empty_like(z), status=status)
    got = sv.adjust_logits(z, R, k, branches, draft, history=history, history_len=ints([1] * R),
                           presence=torch.ones(R, device="cuda"), bias=bias, out=out)["logits"]
    at = torch.arange(R, device="cuda") % (V - 1)
    first = got.view(R, rows, V)
    assert (first[torch.arange(R, device="cuda"), :, at] == -1).all() and not status.any()
    assert (got != 0).sum().item() == R * rows + R * (rows - 1)
"""

CALLS = {
    # a table of 1,366 to 1,373 words beside the marks of a row of 151,936
    "few rows": "adjust(304, 0, 1, 151936, {x}, False)\nadjust(304, 0, 1, 151936, {x}, True)",
    "few rows, biases": "adjust(64, 0, 1, 151936, {x}, False, 16)\nadjust(64, 0, 1, 151936, {x}, True, 16)",
    # in place, slices of 4,096 ids and the numbers of many rows
    "many rows": "adjust(640, {x}, True)",
    "free": """
N = {x}
free, table = torch.full((N,), -1, dtype=torch.int32, device="cuda"), ints([[N - 1, 5], [7, 3]])
got = sv.cache_free(table, ints([9, 16]), ints([1, 0]), free, ints([0]), 8)
assert got["seq_len"].tolist() == [0, 16] and got["free_count"].item() == 2 and free[:3].tolist() == [5, N - 1, -1]
""",
    "compact": """
N = {x}
k = torch.zeros((N, 8, 1, 8), dtype=torch.bfloat16, device="cuda")
v = torch.zeros_like(k)
k[N - 1], k[7], v[5] = 3, 4, 5
got = sv.cache_compact(k, v, ints([[N - 1, 5], [7, 1]]), ints([9, 16]))
assert got["block_table"].tolist() == [[3, 0], [2, 1]] and got["free_count"].item() == N - 4, got["block_table"]
assert (k[3] == 3).all() and (k[2] == 4).all() and (v[0] == 5).all()
""",
}


@pytest.mark.parametrize("name,x", [
    ("few rows", 1366), ("few rows", 1373), ("few rows, biases", 2255), ("few rows, biases", 2259),
    ("many rows", "251, 3, 64, 5"), ("many rows", "108, 7, 64, 5"), ("free", 196608), ("free", 196100), ("compact", 393216),
    ("compact", 391700)])
def test_the_first_call_of_a_process(sv, name, x):
    got = subprocess.run([sys.executable, "-c", HEAD + CALLS[name].format(x=x)], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert got.returncode == 0, got.stderr[-2000:]
