"""adjust_logits with buffers that hold nothing: a step without grammars, a request without room for a history."""
import pytest
import torch

from tests.test_gpu_adjust import Case
from tests.test_gpu_cache import _i32

pytestmark = pytest.mark.gpu


def _bits(t):
    return t.view(torch.int16 if t.dtype is torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,k", [(3, 2), (640, 0), (640, 1)])
def test_a_set_of_no_masks(sv, R, k, dtype):
    """Every row's index is negative; one that is not names a mask above the last."""
    c = Case(R, k, 1, 1003, dtype, masks=None, seed=R + k)
    x, _ = c.logits()
    draft, kw, rows = _i32(c.draft), c.kwargs(), R * (1 + k)
    kw.pop("mask"), kw.pop("mask_row")
    want = sv.adjust_logits(x, R, k, 1, draft, **kw)
    none = torch.empty((0, 32), dtype=torch.int32, device="cuda")
    for index, status in ((-1, 0), (0, 8192)):
        which = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
        which[(1 + k) * 2] = index
        got = sv.adjust_logits(x, R, k, 1, draft, mask=none, mask_row=which, **kw)
        assert torch.equal(_bits(got["logits"]), _bits(want["logits"]))
        more = got["status"] - want["status"]
        assert more[2].item() == status and not more[:2].any() and not more[3:].any()
        y = x.clone()
        got = sv.adjust_logits(y, R, k, 1, draft, mask=none, mask_row=which, out=dict(logits=y, status=got["status"]), **kw)
        assert torch.equal(_bits(y), _bits(want["logits"].contiguous()))
    with pytest.raises(sv.SpecVerifyError):  # neither a mask for each row nor their numbers
        sv.adjust_logits(x, R, k, 1, draft, mask=none, **kw)
    with pytest.raises(sv.SpecVerifyError):  # narrower than the rows
        sv.adjust_logits(x, R, k, 1, draft, mask=none[:, :31].contiguous(), mask_row=which, **kw)


@pytest.mark.parametrize("R,k", [(4, 3), (640, 0)])
def test_a_history_without_room(sv, R, k):
    """Lengths above a width of none are clamped and told."""
    c = Case(R, k, 1, 1003, torch.float32, width=0, seed=R)
    c.history_len[:], c.prompt_len[:] = 0, 0
    _, _, status = c.check(sv)
    assert not status.any()
    c.history_len[1], c.history_len[2], c.prompt_len[3] = 5, -2, 1
    _, _, status = c.check(sv)
    assert status[:4].tolist() == [0, 1024, 1024, 1024]
