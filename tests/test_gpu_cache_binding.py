"""What the binding of the cache operators refuses before it launches anything."""
import pytest
import torch

from tests.test_gpu_cache import Case, _i32

pytestmark = pytest.mark.gpu


# --- refusals ----------------------------------------------------------------------------------------------------
def test_rope_refuses_slots_and_frequencies_on_the_host(sv):
    c = Case([20], [3], 4, 2, 64)
    x, position, slot = c.q[:, :2], _i32([0, 1, 2]), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="freqs"):
        sv.rope_cache(c.q, x, x, position, slot.cuda(), sv.rope_freqs(64, device="cpu"), c.kc, c.vc)
    with pytest.raises(ValueError, match="slot"):
        sv.rope_cache(c.q, x, x, position, slot, sv.rope_freqs(64), c.kc, c.vc)
