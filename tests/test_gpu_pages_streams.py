"""The operators at the two ends of a verify step with stream=, and tensors of another device than the current one."""
import pytest
import torch

from tests.test_gpu_adjust import Case
from tests.test_gpu_cache import _i32, _rope_case
from tests.test_gpu_pages import Pool
from tests.test_gpu_streams import SLEEP, _check_outputs, _check_workspace

pytestmark = pytest.mark.gpu


def _adjust(sv):
    c = Case(6, 3, 2, 3001, torch.bfloat16, seed=1)
    x, draft, kw = c.logits()[0].contiguous(), _i32(c.draft), c.kwargs()

    def call(s):
        got = sv.adjust_logits(x, 6, 3, 2, draft, stream=s, **kw)
        return dict(logits=got["logits"].view(torch.int16), status=got["status"])

    return call


def _pool():
    p = Pool([40, 23, 0, 9, 300], 8, 100, layers=2, seed=2)
    return p, _i32(p.table), _i32(p.seq), _i32(p.free), _i32([p.count])


def _fork(sv):
    p, table, seq, free, count = _pool()
    source = _i32([-1, -1, 1, -1, -1])
    return lambda s: sv.cache_fork(p.k, p.v, table, seq, source, free, count, stream=s)


def _free(sv):
    p, table, seq, free, count = _pool()
    leave = _i32([1, 0, 0, 1, 0])
    return lambda s: sv.cache_free(table, seq, leave, free, count, 8, stream=s)


def _compact(sv):
    p, table, seq, _, _ = _pool()
    return lambda s: sv.cache_compact(p.k, p.v, table, seq, stream=s)


def _norm(sv):
    q, k, v, kc, vc, slot = _rope_case(9, 4, 2, 64, torch.bfloat16)
    position, freqs = _i32(range(9)), sv.rope_freqs(64)
    return lambda s: dict(q=sv.norm_rope_cache(q, k, v, position, slot, freqs, kc, vc, stream=s))


@pytest.mark.parametrize("make", [_adjust, _norm, _fork, _free, _compact])
def test_outputs_belong_to_the_stream(sv, make):
    _check_outputs(make(sv))


def test_compact_workspace_belongs_to_the_stream(sv):
    _check_workspace(_compact(sv), sv.cache_compact_workspace(100))


def test_calls_without_requests_keep_to_the_stream(sv):
    none, table = _i32([]), torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    caches = torch.zeros((8, 8, 1, 8), dtype=torch.bfloat16, device="cuda")
    free, count = _i32(range(8)), _i32([0])
    for call in (lambda s: sv.cache_fork(caches, caches, table, none, none, free, count, stream=s),
                 lambda s: sv.cache_free(table, none, none, free, count, 8, stream=s)):
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            count.fill_(0)
            torch.cuda._sleep(SLEEP)
            count.fill_(7)  # ahead of the call on its stream
        got = call(s)
        torch.cuda.synchronize()
        assert got["free_count"].item() == 7


@pytest.mark.parametrize("make", [_adjust, _norm, _fork, _free, _compact])
def test_tensors_of_another_device_are_refused(sv, monkeypatch, make):
    call = make(sv)
    call(None)
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_cuda_getDevice", lambda: 1)
        with pytest.raises(ValueError, match="current device"):
            call(None)
