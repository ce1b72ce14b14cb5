"""adjust_logits where many requests have few rows each: tables of the ids that rules meet, against the plain 64-bit form."""
import numpy as np
import pytest
import torch

from tests.test_gpu_adjust import Case, _f32
from tests.test_gpu_cache import _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,k,branches,V,width,biases,masks", [
    (700, 0, 1, 1, 3, 1, "own"), (640, 0, 1, 31, 9, 4, "own"), (620, 2, 1, 97, 40, 5, "few"), (330, 1, 1, 9000, 300, 16, "few"),
    (210, 0, 1, 20001, 9000, 3, "own"),     # more ids of a slice than its table has words
    (208, 1, 1, 16500, 50, 6000, None),     # and more biases
    (320, 1, 2, 8200, 0, 0, "own"), (90, 0, 1, 70000, 500, 20, "few"), (160, 2, 1, 32003, 101, 7, None),
    (320, 7, 1, 8203, 130, 9, "few"),       # these in place alone
    (320, 3, 2, 8200, 61, 0, "own")])
def test_few_rows(sv, R, k, branches, V, width, biases, masks, dtype):
    Case(R, k, branches, V, dtype, width, biases, masks, seed=V + R).check(sv)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("stride,offset", [(1031, 0), (1040, 3), (1032, 8), (1025, 5), (1039, 1)])
def test_rows_that_start_anywhere(sv, stride, offset, dtype):
    c = Case(620, 1, 1, 1025, dtype, stride=stride, offset=offset, seed=stride)
    c.check(sv)
    out = torch.empty(c.rows * 1027 + 1, dtype=dtype, device="cuda")[1:].view(c.rows, 1027)[:, :1025]
    c.check(sv, out=dict(logits=out, status=torch.empty(620, dtype=torch.int32, device="cuda")), in_place=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("stride,offset", [(20011, 0), (20016, 7)])
def test_slices_of_rows_that_start_anywhere(sv, stride, offset, dtype):
    """Ids that meet rules on both sides of where slices meet, which is somewhere else in every row."""
    c = Case(120, 1, 1, 20010, dtype, width=200, biases=0, masks="few", stride=stride, offset=offset, seed=offset)
    edges = np.concatenate([np.arange(e - 12, e + 12) for e in range(1024, 20000, 1024)])
    c.history[:] = edges[c.rng.integers(0, len(edges), c.history.shape)]
    c.check(sv)


def test_extreme_values(sv):
    for dtype in (torch.bfloat16, torch.float32):
        c = Case(615, 1, 1, 700, dtype, biases=50, seed=5)
        at = c.rng.random(c.z.shape)
        for i, v in enumerate((np.inf, -np.inf, np.nan, torch.finfo(torch.bfloat16).min, -0.0, 0.0, 1e-38)):
            c.z[(at >= 0.05 * i) & (at < 0.05 * (i + 1))] = v
        c.check(sv)
        c.mask[:] = 0
        got, _, _ = c.check(sv)
        assert torch.isneginf(got["logits"]).all()
        c.mask = None
        c.check(sv)


def test_bad_rules_are_left_out(sv):
    c = Case(615, 2, 1, 300, torch.float32, masks="few", seed=8)
    c.repetition[:4] = 0.0, -1.0, np.nan, np.inf
    c.presence[4:6], c.frequency[6:8] = (np.nan, np.inf), (-np.inf, np.nan)
    c.history[9, 0], c.history_len[9], c.draft[10, 0, 1], c.bias[1][c.bias[0][-2]] = 300, 60, 2 ** 31 - 1, -2 ** 31
    c.mask_row[3 * 20 + 2] = 3
    c.history_len[30:34] = -1, 61, 60, 2 ** 31 - 1
    c.prompt_len[30:34] = 0, 0, 61, 7
    _, _, status = c.check(sv)
    assert status[:8].tolist() == [4096] * 8 and status[8] == 0
    assert (status[[9, 10, 614]] & 1).all() and status[20] == 8192 and (status[30:34] == 1024).all()
    c = Case(615, 0, 1, 300, torch.float32, biases=9, seed=11)
    start = c.bias[0]
    start[0], start[2], start[-1] = -3, start[1] - 1, len(c.bias[1]) + 5
    _, _, status = c.check(sv)
    assert (status[[0, 1, 614]] == 1024).all()


def test_the_same_id_twice(sv):
    c = Case(613, 1, 2, 64, torch.float32, width=3000, biases=0, seed=12)
    c.history[:], c.draft[:] = 5, 5
    c.history[:, ::7] = 6
    start = np.zeros(614, np.int32)
    start[1:], start[-1] = 4, 9
    c.bias = (start, np.array([5, 9, 5, 5, 7, 7, 6, 7, 6], np.int32), np.arange(9).astype(np.float32) - 4)
    c.check(sv)


def test_histories_that_start_anywhere(sv):
    for width in (8193, 8195, 2):
        Case(205, 0, 1, 20000, torch.bfloat16, width=width, biases=2, masks=None, seed=width).check(sv)


def test_results_do_not_depend_on_the_batch(sv):
    """A request alone has the bits it has among many, in and out of place, with a vocabulary of several of the longest
    slices."""
    R, V, width = 310, 262144 * 2 + 17, 6000
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randn((R, V), generator=g, device="cuda", dtype=torch.bfloat16)
    history = torch.randint(0, V, (R, width), generator=g, device="cuda", dtype=torch.int32)
    length = torch.randint(0, width + 1, (R,), generator=g, device="cuda", dtype=torch.int32)
    rules = dict(history=history, history_len=length, prompt_len=length // 2, repetition=torch.rand(R, device="cuda") + 0.5,
                 presence=torch.rand(R, device="cuda"), frequency=torch.rand(R, device="cuda"),
                 mask=torch.randint(-2 ** 31, 2 ** 31, (R, -(-V // 32)), generator=g, device="cuda", dtype=torch.int32))
    draft = torch.empty((R, 1, 0), dtype=torch.int32, device="cuda")
    many = sv.adjust_logits(z, R, 0, 1, draft, **rules)["logits"].view(torch.int16)
    assert not torch.equal(many, z.view(torch.int16))
    for r in (0, 1, 200, 309):
        one = {n: x[r:r + 1].contiguous() for n, x in rules.items()}
        alone = sv.adjust_logits(z[r:r + 1], 1, 0, 1, draft[:1], **one)["logits"]
        assert torch.equal(alone[0].view(torch.int16), many[r])
    sv.adjust_logits(z, R, 0, 1, draft, out=dict(logits=z), **rules)
    assert torch.equal(z.view(torch.int16), many)


def test_long_histories(sv):
    """The longest history of one request among many."""
    R, V = 205, 20000
    history = torch.zeros((R, 524287), dtype=torch.int32, device="cuda")
    history[:, ::2] = torch.arange(262144, dtype=torch.int32, device="cuda") % 10007
    history[:, 1::2] = 10008
    length = torch.arange(R, dtype=torch.int32, device="cuda")
    length[7] = 524287
    freq = torch.full((R,), 2.0 ** -12, device="cuda")
    z = torch.zeros((R, V), device="cuda")
    got = sv.adjust_logits(z, R, 0, 1, history=history, history_len=length, frequency=freq)
    want = torch.zeros((R, V), dtype=torch.float64)
    for r in range(R):
        want[r] -= torch.bincount(history[r, :length[r]].long().cpu(), minlength=V) * 2.0 ** -12
    assert torch.equal(got["logits"].double().cpu(), want) and not got["status"].any()  # all of it is exact in fp32


def test_captured_and_replayed_on_another_stream(sv):
    c = Case(640, 1, 1, 3001, torch.bfloat16, width=200, seed=18)
    x, _ = c.logits()
    x = x.contiguous()
    kw, draft = c.kwargs(), _i32(c.draft)
    want = sv.adjust_logits(x, 640, 1, 1, draft, **kw)["logits"]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sv.adjust_logits(x, 640, 1, 1, draft, **kw)["logits"]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(2):
            got.zero_()
            g.replay()
        other = sv.adjust_logits(x, 640, 1, 1, draft, **kw)["logits"]
    side.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and torch.equal(other.view(torch.int16), want.view(torch.int16))


def test_rows_behind_the_last_stay(sv):
    x = torch.randn((623, 100), device="cuda")
    x[620:] = 5.0
    rep = _f32(np.full(620, 1.5))
    history = _i32(np.arange(620)[:, None] % 100)
    sv.adjust_logits(x, 620, 0, 1, out=dict(logits=x), history=history, history_len=_i32([1] * 620), repetition=rep)
    assert (x[620:] == 5.0).all()
