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


def _wrong(t):
    """Tensors that cannot stand for an output like t."""
    flat = t.reshape(-1)
    yield flat[:-1].clone()                                        # an entry short
    yield torch.empty(t.shape, dtype=t.dtype)                      # on the host
    yield torch.empty(t.shape, dtype=torch.float64, device="cuda")  # another type
    if flat.numel() > 1:
        yield torch.empty(2 * flat.numel(), dtype=t.dtype, device="cuda")[::2]  # strided


def test_outputs_without_room_are_refused(sv):
    R, T, words, k = 2, 9, 2, 3
    c = Case([20, 7], [5, 4], 4, 2, 64)
    seq, new, free, count = _i32([20, 7]), _i32([5, 4]), _i32(range(40)), _i32([40])
    parent = _i32([-1, 0, 1, 2, 3, -1, 0, 1, 2])
    table = torch.zeros((R, 8), dtype=torch.int32, device="cuda")
    caches = [torch.zeros((40, 16, 2, 64), dtype=c.dtype, device="cuda") for _ in range(2)]

    def tables(out=None):
        return sv.step_tables(seq, new, table, free, count, 16, T, parent=parent, mask_words=words, out=out)

    def attend(out=None):
        return sv.tree_attention(c.q, c.kc, c.vc, c.table, _i32(c.kv), _i32(c.cu), 5, with_lse=True, out=out)

    def commit(out=None):
        return sv.cache_commit(*caches, table, seq, _i32([25, 11]), _i32([0, 5, 9]), _i32([1, 2]), k, free, count,
                               out=out)

    for call in (tables, attend, commit):
        out = call()
        out.setdefault("status", torch.empty(R, dtype=torch.int32, device="cuda"))
        for name, t in out.items():
            if name == "out":
                continue  # heads may be strided: the library checks them
            for bad in _wrong(t):
                with pytest.raises(ValueError, match=name):
                    call(dict(out, **{name: bad}))
        roomy = {name: t if name == "out" else torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
                 for name, t in out.items()}
        assert call(roomy) is roomy
        call({name: t for name, t in out.items() if name != "status"})  # asked for or not
    with pytest.raises(ValueError, match="mask"):  # room enough, in rows of another width
        tables(dict(tables(), mask=torch.empty((T, words + 1), dtype=torch.int32, device="cuda")))
    with pytest.raises(sv.SpecVerifyError):
        attend(dict(out=torch.empty_like(c.q)[:-1]))
    with pytest.raises(ValueError, match="workspace"):
        sv.tree_attention(c.q, c.kc, c.vc, c.table, _i32(c.kv), _i32(c.cu), 5,
                          workspace=torch.empty(1 << 26, dtype=torch.uint8))
    torch.cuda.synchronize()


def test_tensors_of_another_device_are_refused(sv, monkeypatch):
    """Where the current device is another than the tensors', nothing is launched."""
    c = Case([20], [3], 4, 2, 64)
    seq, new, free, count = _i32([20]), _i32([3]), _i32(range(8)), _i32([8])
    table = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    kv, cu, slot, freqs = _i32(c.kv), _i32(c.cu), torch.zeros(3, dtype=torch.int64, device="cuda"), sv.rope_freqs(64)
    x, nb = c.q[:, :2].contiguous(), c.kc.shape[0]
    calls = [lambda: sv.step_tables(seq, new, table, free, count, 16, 3),
             lambda: sv.rope_cache(c.q, x, x, cu.new_zeros(3), slot, freqs, c.kc, c.vc),
             lambda: sv.tree_attention(c.q, c.kc, c.vc, c.table, kv, cu, 3),
             lambda: sv.cache_commit(c.kc, c.vc, c.table, seq, kv, cu, new, 2, free.new_zeros(nb), count)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_cuda_getDevice", lambda: 1)
        for call in calls:
            with pytest.raises(ValueError, match="current device"):
                call()
