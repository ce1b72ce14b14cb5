"""adjust_logits with slices of several regions (requests of nine rows and more, in numbers that fill the GPU): in place, to rows
that start alike and to rows that start differently, and from two threads with different amounts of shared memory."""
import threading

import numpy as np
import pytest
import torch

from tests.test_gpu_adjust import Case
from tests.test_gpu_cache import _i32

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


def _apart(c, pad, start):
    """An output whose rows start elsewhere within 16 bytes than those of the input, in rows of V + pad entries."""
    wide = c.V + pad
    y = torch.empty(c.rows * wide + start, dtype=c.dtype, device="cuda")[start:].view(c.rows, wide)[:, :c.V]
    return dict(logits=y, status=torch.empty(c.R, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,k,branches,V,width,biases,masks,stride,offset", [
    (80, 8, 1, 32003, 700, 20, "few", None, 0), (80, 8, 1, 32000, 61, 0, "own", None, 0),
    (80, 8, 1, 32003, 5000, 2000, None, None, 0),       # more biases than 16 bits count
    (310, 3, 4, 8203, 90, 9, "own", 8208, 3), (160, 10, 1, 17000, 300, 5, "few", 17011, 5),
    (17, 9, 1, 151936, 4500, 300, "few", None, 0), (320, 2, 8, 4090, 0, 0, "few", 4097, 1)])
def test_several_regions(sv, R, k, branches, V, width, biases, masks, stride, offset, dtype):
    c = Case(R, k, branches, V, dtype, width, biases, masks, seed=V + k, stride=stride, offset=offset)
    c.check(sv)
    c.check(sv, out=_apart(c, 3, 1), in_place=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("stride,offset", [(16391, 0), (16392, 7), (16400, 0), (16385, 2)])
def test_ids_where_regions_meet(sv, stride, offset, dtype):
    c = Case(160, 9, 1, 16384, dtype, width=250, biases=0, masks="few", stride=stride, offset=offset, seed=stride)
    edges = np.concatenate([np.arange(max(e - 12, 0), min(e + 12, 16384)) for e in range(0, 16385, 512)])
    c.history[:] = edges[c.rng.integers(0, len(edges), c.history.shape)]
    c.draft[:] = edges[c.rng.integers(0, len(edges), c.draft.shape)]
    c.check(sv)
    c.check(sv, out=_apart(c, 1, 3), in_place=False)


@pytest.mark.parametrize("dtype", DTYPES)
def test_extreme_values(sv, dtype):
    c = Case(160, 8, 1, 16390, dtype, biases=50, seed=5)
    at = c.rng.random(c.z.shape)
    for i, v in enumerate((np.inf, -np.inf, np.nan, torch.finfo(torch.bfloat16).min, -0.0, 0.0, 1e-38)):
        c.z[(at >= 0.05 * i) & (at < 0.05 * (i + 1))] = v
    c.check(sv)
    c.mask[:] = 0
    got, _, _ = c.check(sv)
    assert torch.isneginf(got["logits"]).all()
    c.mask = None
    c.check(sv)


def test_crowded_regions(sv):
    """Every id of a slice met by a rule, one of them by every token."""
    c = Case(160, 8, 1, 16384, torch.bfloat16, width=4096, biases=0, masks="few", seed=6)
    c.history[:] = np.arange(4096) + 4090
    c.history[::2, ::3] = 4096
    c.history_len[:] = 4096
    c.draft[:] = 4096
    c.check(sv)


def _at_once(sv, cases):
    args, wants, wrong = [], [], []

    def call(i):
        x, draft, kw = args[i]
        return sv.adjust_logits(x, cases[i].R, cases[i].k, 1, draft, **kw)["logits"].view(torch.int16)

    for i, c in enumerate(cases):
        args.append((c.logits()[0].contiguous(), _i32(c.draft), c.kwargs()))
        wants.append(call(i))
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(100):
                    got = call(i)
                torch.cuda.current_stream().synchronize()
                if not torch.equal(got, wants[i]):
                    wrong.append(i)
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_threads_with_one_kernel_and_other_slices(sv):
    """Slices of 2,048 and of 4,096 ids: 51 and 68 KB a thread block."""
    _at_once(sv, [Case(64, 4, 1, 32003, torch.bfloat16, seed=24), Case(80, 8, 1, 32003, torch.bfloat16, seed=25)])


def test_threads_with_one_kernel_and_other_tables(sv):
    """Tables of 2,000 and of 4,000 words beside the marks of 140,001 ids: 51 and 67 KB a thread block."""
    _at_once(sv, [Case(310, 0, 1, 140001, torch.bfloat16, width=w, biases=0, masks=None, seed=w) for w in (2000, 4000)])
