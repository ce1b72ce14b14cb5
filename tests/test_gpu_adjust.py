"""adjust_logits on the GPU against the plain 64-bit form, within fp32's roundings and one to the rows' type."""
import numpy as np
import pytest
import torch

from tests import pages_plain as plain
from tests.test_gpu_cache import _i32

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}  # fp32's own rounding is in the plain form's bound
# below the normal range half a step is absolute: 2^-150 for each of fp32's four, 2^-134 for bf16's one
TINY = {torch.bfloat16: 2.0 ** -134 + 2.0 ** -148, torch.float32: 2.0 ** -148}


def _f32(a):
    return torch.tensor(np.asarray(a, np.float32)).cuda()


class Case:
    """Random rules for R requests; everything may be spoiled before `check`."""

    def __init__(self, R, k, branches, V, dtype, width=60, biases=5, masks="own", seed=0, stride=None, offset=0):
        rng = np.random.default_rng(seed)
        self.R, self.k, self.branches, self.V, self.dtype, self.rng = R, k, branches, V, dtype, rng
        self.rows = R * (1 + branches * k)
        self.stride = V if stride is None else stride
        self.offset = offset  # entries that the first row starts behind its allocation
        self.z = rng.normal(0, 3, (self.rows, V)).astype(np.float32)
        few = rng.integers(0, V, 12)
        pick = lambda *s: np.where(rng.random(s) < 0.7, few[rng.integers(0, 12, s)], rng.integers(0, V, s)).astype(np.int32)  # noqa: E731
        self.draft = pick(R, branches, k)
        self.history, self.history_len = pick(R, width), rng.integers(0, width + 1, R).astype(np.int32)
        self.history_len[0] = width
        if R > 2:
            self.history_len[1] = 0
        self.prompt_len = (self.history_len * rng.random(R)).astype(np.int32)
        self.repetition = rng.uniform(0.7, 1.5, R).astype(np.float32)
        self.presence = rng.uniform(-0.5, 0.7, R).astype(np.float32)
        self.frequency = rng.uniform(-0.1, 0.3, R).astype(np.float32)
        self.bias = self.mask = self.mask_row = None
        if biases:
            m = rng.integers(0, biases + 1, R)
            m[-1] = biases
            ids = np.concatenate([rng.choice(V, min(x, V), replace=False) for x in m]).astype(np.int32)
            m = np.minimum(m, V)
            values = rng.normal(0, 2, len(ids)).astype(np.float32)
            values[rng.random(len(ids)) < 0.2] = -np.inf
            self.bias = (np.concatenate([[0], np.cumsum(m)]).astype(np.int32), ids, values)
        if masks:
            n = self.rows if masks == "own" else 3
            self.mask = rng.integers(-2 ** 31, 2 ** 31, (n, -(-V // 32))).astype(np.int32)
            self.mask[rng.random(self.mask.shape) < 0.3] = -1
            self.mask[rng.random(self.mask.shape) < 0.3] = 0
            if masks != "own":
                self.mask_row = rng.integers(-1, 3, self.rows).astype(np.int32)

    def kwargs(self):
        d = lambda x, f: None if x is None else f(x)  # noqa: E731
        return dict(history=d(self.history, _i32), history_len=d(self.history_len, _i32), prompt_len=d(self.prompt_len, _i32),
                    repetition=d(self.repetition, _f32), presence=d(self.presence, _f32), frequency=d(self.frequency, _f32),
                    bias=None if self.bias is None else (_i32(self.bias[0]), _i32(self.bias[1]), _f32(self.bias[2])),
                    mask=d(self.mask, _i32), mask_row=d(self.mask_row, _i32))

    def logits(self):
        room = torch.full((self.offset + self.rows * self.stride + 64,), 7.0, dtype=self.dtype, device="cuda")
        x = room[self.offset:self.offset + self.rows * self.stride].view(self.rows, self.stride)[:, :self.V]
        x.copy_(torch.from_numpy(self.z))
        return x, room

    def check(self, sv, in_place=True, out=None):
        x, room = self.logits()
        before = x.clone()
        raw = x.double().cpu().numpy()
        with np.errstate(invalid="ignore", over="ignore"):
            want, err, status = plain.adjust(raw, self.R, self.k, self.branches, self.draft, self.history, self.history_len,
                                             self.prompt_len, self.repetition, self.presence, self.frequency, self.bias,
                                             self.mask, self.mask_row)
        draft, kw = _i32(self.draft), self.kwargs()
        got = sv.adjust_logits(x, self.R, self.k, self.branches, draft, out=out, **kw)
        torch.cuda.synchronize()
        assert torch.equal(x, before) or not torch.isfinite(before).all()
        self.compare(got, want, err, status)
        if in_place:
            gap = room.clone()
            res = dict(logits=x, status=torch.full((self.R,), -1, dtype=torch.int32, device="cuda"))
            sv.adjust_logits(x, self.R, self.k, self.branches, draft, out=res, **kw)
            torch.cuda.synchronize()
            same = got["logits"].view(torch.int16 if self.dtype is torch.bfloat16 else torch.int32)
            assert torch.equal(x.contiguous().view(same.dtype), same)  # the bits of the other form
            x.copy_(before)
            bits = torch.int16 if self.dtype is torch.bfloat16 else torch.int32
            assert torch.equal(room.view(bits), gap.view(bits))  # nothing but the rows
        return got, want, status

    def compare(self, got, want, err, status):
        y = got["logits"].double().cpu().numpy()
        with np.errstate(invalid="ignore"):
            tol = err + HALF[self.dtype] * (np.abs(want) + err) + TINY[self.dtype]
            bad = ~((np.abs(y - want) <= tol) | (y == want) | (np.isnan(y) & np.isnan(want)))
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[:5], y[bad][:5], want[bad][:5])
        np.testing.assert_array_equal(got["status"].cpu().numpy(), status)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,k,branches,V,width,biases,masks", [
    (1, 0, 1, 1, 3, 1, "own"), (1, 0, 1, 151936, 777, 0, None), (3, 1, 1, 31, 9, 4, "own"), (5, 8, 1, 4096, 300, 16, "few"),
    (2, 16, 2, 32003, 500, 100, "own"), (7, 4, 8, 1000, 60, 3, "few"), (40, 3, 1, 8191, 40, 0, "own"),
    (3, 256, 8, 257, 1500, 7, "few"), (200, 0, 1, 5000, 20, 5, None), (2, 3, 1, 1023, 0, 0, "own"),
    (1, 5, 1, 200001, 4000, 300, "few"), (30, 2, 1, 16385, 100, 2000, None),
    (40, 1, 1, 5000, 60, 5000, "few"),      # more biases than 16 bits count
    (3, 2, 1, 9001, 8195, 9, "own"),        # long rows of history that start anywhere
    (40, 1, 1, 140001, 600, 20, "few"),     # the wide slices of one or two rows
    (160, 0, 1, 40008, 4100, 3, "own")])
def test_adjust(sv, R, k, branches, V, width, biases, masks, dtype):
    Case(R, k, branches, V, dtype, width, biases, masks, seed=V + R).check(sv)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("stride,offset", [(1031, 0), (1040, 3), (1032, 8), (1025, 5)])
def test_rows_that_start_anywhere(sv, stride, offset, dtype):
    c = Case(4, 2, 2, 1025, dtype, stride=stride, offset=offset, seed=stride)
    c.check(sv)
    # rows of the two matrices that start differently within a vector
    out = torch.empty(c.rows * 1027 + 1, dtype=dtype, device="cuda")[1:].view(c.rows, 1027)[:, :1025]
    c.check(sv, out=dict(logits=out, status=torch.empty(4, dtype=torch.int32, device="cuda")), in_place=False)


def test_extreme_values(sv):
    """Infinities and NaN in seen, unseen and masked places, and the lowest value of the type."""
    for dtype in (torch.bfloat16, torch.float32):
        c = Case(6, 2, 1, 700, dtype, biases=50, seed=5)
        at = c.rng.random(c.z.shape)
        for i, v in enumerate((np.inf, -np.inf, np.nan, torch.finfo(torch.bfloat16).min, -0.0, 0.0, 1e-38)):
            c.z[(at >= 0.05 * i) & (at < 0.05 * (i + 1))] = v
        c.check(sv)
        c.mask[:] = 0  # nothing is allowed
        got, _, _ = c.check(sv)
        assert torch.isneginf(got["logits"]).all()
        c.mask = None
        c.check(sv)


def test_untouched_entries_keep_their_bits(sv):
    z = torch.full((2, 500), float("nan"), device="cuda").view(torch.int32)
    z += torch.arange(500, dtype=torch.int32, device="cuda") + 77  # NaN of every kind
    z = z.view(torch.float32)
    got = sv.adjust_logits(z, 2, 0, 1, repetition=_f32([1.2, 1.2]), history=_i32([[1, 2], [499, 0]]), history_len=_i32([2, 2]))
    rest = [i for i in range(500) if i not in (1, 2)]
    assert torch.equal(got["logits"].view(torch.int32)[0, rest], z.view(torch.int32)[0, rest])


def test_bad_rules_are_left_out(sv):
    c = Case(9, 3, 1, 300, torch.float32, masks="few", seed=8)
    c.repetition[:4] = 0.0, -1.0, np.nan, np.inf
    c.presence[4:6], c.frequency[6:8] = (np.nan, np.inf), (-np.inf, np.nan)
    _, _, status = c.check(sv)
    assert status.tolist() == [4096] * 8 + [0]
    c = Case(6, 3, 1, 300, torch.bfloat16, masks="few", seed=9)
    c.history_len[:] = 60
    c.history[0, 7], c.history[1, 59], c.draft[2, 0, 1], c.bias[1][c.bias[0][3]] = 300, -1, 2 ** 31 - 1, -2 ** 31
    c.mask_row[17] = 3
    _, _, status = c.check(sv)
    assert status[0] == status[1] == status[2] == 1 and status[4] & 8192
    c = Case(5, 0, 1, 300, torch.float32, seed=10)
    c.history_len[:] = -1, 61, 60, 30, 2 ** 31 - 1
    c.prompt_len[:] = 0, 0, 61, -5, 7
    _, _, status = c.check(sv)
    assert (status == 1024).all()
    c = Case(4, 0, 1, 300, torch.float32, biases=9, seed=11)
    start = c.bias[0]
    start[0], start[2], start[4] = -3, start[1] - 1, len(c.bias[1]) + 5
    _, _, status = c.check(sv)
    assert (status[[0, 1, 3]] == 1024).all()


def test_the_same_id_twice(sv):
    """Twice in the biases: the last entry counts.  A thousand times in history and drafts: a thousand counts."""
    c = Case(3, 16, 8, 64, torch.float32, width=3000, seed=12)
    c.history[:], c.draft[:] = 5, 5
    c.history[:, ::7] = 6
    c.bias = (np.array([0, 4, 4, 9], np.int32), np.array([5, 9, 5, 5, 7, 7, 6, 7, 6], np.int32),
              np.arange(9).astype(np.float32) - 4)
    c.check(sv)


def test_rules_one_at_a_time(sv):
    for name in ("history", "prompt_len", "repetition", "presence", "frequency", "bias", "mask"):
        c = Case(3, 2, 2, 2050, torch.bfloat16, seed=13)
        setattr(c, name, None)
        c.check(sv)
        c = Case(3, 2, 2, 2050, torch.bfloat16, masks="few", seed=13)
        if name != "mask":
            setattr(c, name, None)
        c.check(sv)
        c = Case(3, 2, 2, 2050, torch.bfloat16, seed=14)
        for other in ("prompt_len", "repetition", "presence", "frequency", "bias", "mask"):
            if other != name:
                setattr(c, other, None)
        c.check(sv)


def test_a_long_history(sv):
    c = Case(1, 1, 1, 40000, torch.float32, width=524287, biases=0, masks=None, seed=15)
    c.history_len[:], c.prompt_len[:] = 524287, 0
    c.history[0, 1000:] = 17
    c.frequency[:] = 0.001
    c.check(sv)


def test_results_do_not_depend_on_the_batch(sv):
    """Alone, with other slices and groups of rows, a request has the bits it has among many."""
    c = Case(64, 4, 1, 32003, torch.bfloat16, width=400, seed=16)
    x, _ = c.logits()
    kw, draft = c.kwargs(), _i32(c.draft)
    many = sv.adjust_logits(x, 64, 4, 1, draft, **kw)["logits"]
    for r in (0, 1, 63):
        b0, b1 = int(c.bias[0][r]), int(c.bias[0][r + 1])
        one = dict(bias=(_i32([0, b1 - b0]), kw["bias"][1][b0:b1].contiguous(), kw["bias"][2][b0:b1].contiguous()),
                   mask=kw["mask"][5 * r:5 * r + 5].contiguous())
        one.update({n: kw[n][r:r + 1].contiguous() for n in ("history", "history_len", "prompt_len", "repetition",
                                                             "presence", "frequency")})
        alone = sv.adjust_logits(x[5 * r:5 * r + 5], 1, 4, 1, draft[r:r + 1].contiguous(), **one)["logits"]
        assert torch.equal(alone.view(torch.int16), many[5 * r:5 * r + 5].view(torch.int16))


def test_rows_past_32_bits(sv):
    """Offsets of rows past 2^32 bytes and 2^32 entries, in place and to columns beside them."""
    for dtype, stride in ((torch.bfloat16, 2 ** 31 + 24), (torch.float32, 2 ** 30 + 12)):
        c = Case(1, 2, 1, 700, dtype, seed=20)
        room = torch.empty(2 * stride + 2000, dtype=dtype, device="cuda")
        x, y = (room[o:].as_strided((3, 700), (stride, 1)) for o in (0, 1000))
        x.copy_(torch.from_numpy(c.z))
        raw = x.double().cpu().numpy()
        want, err, status = plain.adjust(raw, 1, 2, 1, c.draft, c.history, c.history_len, c.prompt_len, c.repetition,
                                         c.presence, c.frequency, c.bias, c.mask)
        for out in (y, x):
            got = sv.adjust_logits(x, 1, 2, 1, _i32(c.draft), out=dict(logits=out, status=_i32([7])), **c.kwargs())
            torch.cuda.synchronize()
            c.compare(got, want, err, status)
        del room, x, y
        torch.cuda.empty_cache()


def test_outputs_that_meet_the_rows_are_refused(sv):
    c = Case(2, 1, 1, 100, torch.float32, seed=21)
    room = torch.zeros((6, 300), device="cuda")
    x, draft, kw = room[:4, :100], _i32(c.draft), c.kwargs()
    x.copy_(torch.from_numpy(c.z))
    want = sv.adjust_logits(x, 2, 1, 1, draft, **kw)["logits"]
    for bad in (room[:4, 50:150], room[1:5, :100], room[1:5, 250:], room.view(-1)[100:].as_strided((4, 100), (100, 1))):
        if bad.shape[1] == 100:
            with pytest.raises(sv.SpecVerifyError):
                sv.adjust_logits(x, 2, 1, 1, draft, out=dict(logits=bad), **kw)
    for good in (room[:4, 100:200], room[2:, 200:]):
        got = sv.adjust_logits(x, 2, 1, 1, draft, out=dict(logits=good), **kw)["logits"]
        assert torch.equal(got, want)


def test_rows_behind_the_last_stay(sv):
    c = Case(2, 1, 1, 100, torch.float32, seed=17)
    x, _ = c.logits()
    more = torch.cat([x, torch.full((3, 100), 5.0, device="cuda")])
    sv.adjust_logits(more, 2, 1, 1, _i32(c.draft), out=dict(logits=more), **c.kwargs())
    assert (more[4:] == 5.0).all()
    assert sv.adjust_logits(more, 2, 1, 1, _i32(c.draft), **c.kwargs())["logits"].shape == (4, 100)


def test_no_requests(sv):
    got = sv.adjust_logits(torch.empty((0, 50), device="cuda"), 0, 3, 1, torch.empty((0, 1, 3), dtype=torch.int32, device="cuda"))
    assert got["logits"].shape == (0, 50) and got["status"].numel() == 0


def test_captured_and_replayed(sv):
    c = Case(5, 3, 2, 3001, torch.bfloat16, seed=18)
    x, _ = c.logits()
    kw, draft = c.kwargs(), _i32(c.draft)
    want = sv.adjust_logits(x, 5, 3, 2, draft, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sv.adjust_logits(x, 5, 3, 2, draft, **kw)
    got["logits"].zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got["logits"].view(torch.int16), want["logits"].view(torch.int16))


def test_a_replayed_graph_takes_new_rules(sv):
    c, d = (Case(5, 3, 2, 3001, torch.bfloat16, seed=x) for x in (22, 23))
    x, _ = c.logits()
    kw, draft = c.kwargs(), _i32(c.draft)
    call = lambda: sv.adjust_logits(x, 5, 3, 2, draft, **kw)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    d.bias = None
    c.bias = None
    for name, t in d.kwargs().items():
        if name != "bias" and t is not None:
            kw[name].copy_(t)
    kw["bias"][0].zero_()
    draft.copy_(_i32(d.draft)), x.copy_(d.logits()[0])
    g.replay()
    torch.cuda.synchronize()
    want, err, status = plain.adjust(x.double().cpu().numpy(), 5, 3, 2, d.draft, d.history, d.history_len, d.prompt_len,
                                     d.repetition, d.presence, d.frequency, None, d.mask)
    d.compare(got, want, err, status)


def test_threads_with_slices_of_other_sizes(sv):
    """Calls from two threads at once, which need different amounts of shared memory."""
    import threading

    cases = [Case(1, 2, 1, 700, torch.bfloat16, seed=24), Case(64, 2, 1, 32003, torch.bfloat16, seed=25)]
    args, wants, wrong = [], [], []
    for c in cases:
        args.append((c.logits()[0].contiguous(), _i32(c.draft), c.kwargs()))
        wants.append(sv.adjust_logits(args[-1][0], c.R, 2, 1, args[-1][1], **args[-1][2])["logits"])
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(200):
                    got = sv.adjust_logits(args[i][0], cases[i].R, 2, 1, args[i][1], **args[i][2])["logits"]
                torch.cuda.current_stream().synchronize()
                if not torch.equal(got.view(torch.int16), wants[i].view(torch.int16)):
                    wrong.append(i)
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_refusals(sv):
    c = Case(2, 3, 1, 100, torch.float32, seed=19)
    x, _ = c.logits()
    draft, kw = _i32(c.draft), c.kwargs()
    call = lambda logits=x, draft=draft, out=None, **more: sv.adjust_logits(logits, 2, 3, 1, draft, out=out, **dict(kw, **more))  # noqa: E731
    call()
    for bad in (x[:7], x.half(), x.cpu(), x[:, ::2], x.flatten()):
        with pytest.raises((ValueError, TypeError)):
            call(logits=bad)
    for bad in (None, draft.long(), draft.cpu(), draft[:, :, :2].contiguous()):
        with pytest.raises(ValueError, match="draft"):
            call(draft=bad)
    for name in ("repetition", "presence", "frequency"):
        for bad in (kw[name].double(), kw[name].cpu(), kw[name][:1]):
            with pytest.raises(ValueError, match=name):
                call(**{name: bad})
    with pytest.raises(ValueError, match="history"):
        call(history_len=None)
    with pytest.raises(ValueError, match="history_len"):
        call(history_len=kw["history_len"][:1])
    with pytest.raises(ValueError, match="start"):
        call(bias=(kw["bias"][0][:2], *kw["bias"][1:]))
    with pytest.raises(ValueError, match="values"):
        call(bias=(*kw["bias"][:2], kw["bias"][2][1:]))
    with pytest.raises(sv.SpecVerifyError):
        call(mask=kw["mask"][:, :3].contiguous())  # narrower than the rows
    with pytest.raises(sv.SpecVerifyError):
        call(mask=kw["mask"][:5].contiguous())     # neither a mask for each row nor their numbers
    with pytest.raises(ValueError, match="mask_row"):
        call(mask_row=_i32([0]))
    with pytest.raises(ValueError, match="mask_row"):
        call(mask=None, mask_row=_i32([0] * 8))
    status = torch.empty(2, dtype=torch.int32, device="cuda")
    with pytest.raises(sv.SpecVerifyError):
        call(out=dict(logits=torch.empty_like(x, dtype=torch.bfloat16), status=status))
    with pytest.raises(ValueError, match="logits"):
        call(out=dict(logits=torch.empty_like(x)[:7], status=status))
    with pytest.raises(ValueError, match="status"):
        call(out=dict(logits=torch.empty_like(x), status=status[:1]))
    torch.cuda.synchronize()
