"""serving_sampler_gb300 -- Python binding of the specverify C library.

The binding only marshals arguments: it turns torch tensors into raw device
pointers and sizes, calls the C entry points of ``libspecverify.so`` through
ctypes on the current CUDA stream, and raises on a non-zero return code.
Every step of verification runs in the library's CUDA kernels; there is no
fallback.  If the library has not been built, ``load()`` raises.

Entry points (same names as the C ABI in include/specverify.h):
  verify_greedy, verify_sample, cfg_merge_sample, accept_scan
  step_tables, rope_cache (with rope_freqs), tree_attention, cache_commit: the
  cache side of a verify step

Every call runs on the current stream, or on ``stream=``.  What it allocates by
itself belongs to that stream; its inputs must be ready on it and stay alive
until it has read them, as with any work on a stream that is not their own.
"""
from __future__ import annotations

import ctypes as C
import os

from . import _build

LIB_PATH = _build.LIB

SV_BF16, SV_F32, SV_F16 = 0, 1, 2
ST_TOKEN_RANGE, ST_BAD_LOGITS, ST_OFF_SUPPORT, ST_RESIDUAL_ZERO = 1, 2, 4, 8
ST_BAD_TEMP, ST_BAD_D2T, ST_TIMEOUT, ST_POOL_FULL = 16, 32, 64, 128
ST_NO_BLOCKS, ST_BAD_TREE, ST_BAD_LENGTH, ST_BAD_BLOCK = 256, 512, 1024, 2048
MAX_K, MAX_S, MAX_NGRAM, MAX_POOL = 256, 16, 64, 1 << 24
MAX_HEAD_DIM, MAX_GROUP, MAX_TREE = 128, 128, 2049
ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_BY_DIM, ROPE_BY_TURNS = 0, 1, 2, 3, 4

# kernels launched by one call of each entry point (reported by the benchmark)
# kernels one call launches: verify_sample with a prebuilt d2t plan (or the identity map)
# launches 2, and 2 more when it builds the plan itself; d2t_plan launches 2
LAUNCHES = {"verify_greedy": 2, "verify_greedy_top2": 2, "infer_modality": 2, "pool_append": 1, "pool_lookup": 1, "suffix_append": 1, "verify_sample": 2, "verify_sample_plan_in_call": 4, "d2t_plan": 2,
            "cfg_merge_sample": 2, "accept_scan": 1, "step_tables": 1, "rope_cache": 1, "tree_attention": 2,
            "cache_commit": 1}


class SpecVerifyError(RuntimeError):
    def __init__(self, code: int, text: str):
        super().__init__(f"specverify error {code}: {text}")
        self.code = code


class SvRows(C.Structure):
    _fields_ = [("data", C.c_void_p), ("dtype", C.c_int32), ("width", C.c_int32), ("row_stride", C.c_int64)]


class SvKvCache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("dtype", C.c_int32), ("num_blocks", C.c_int32),
                ("block_size", C.c_int32), ("kv_heads", C.c_int32), ("head_dim", C.c_int32), ("layers", C.c_int32),
                ("block_stride", C.c_int64), ("token_stride", C.c_int64), ("head_stride", C.c_int64),
                ("layer_stride", C.c_int64)]


class SvHeads(C.Structure):
    _fields_ = [("data", C.c_void_p), ("dtype", C.c_int32), ("tokens", C.c_int32), ("heads", C.c_int32),
                ("head_dim", C.c_int32), ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


_lib = None
torch = None  # set by load()


def load(path: str | None = None):
    """Load libspecverify.so (built in-tree by ``_build.build()``)."""
    global _lib, torch
    if _lib is not None:
        return _lib
    import torch  # the calls below the loader use the module's name: an import statement in each costs more

    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the CUDA library first (python -c 'import __graft_entry__ as g; g.build()')"
        )
    lib = C.CDLL(path)
    P, i32, sz, f32 = C.c_void_p, C.c_int32, C.c_size_t, C.c_float
    lib.sv_status_string.argtypes = [C.c_int]
    lib.sv_status_string.restype = C.c_char_p
    lib.sv_verify_greedy_workspace.argtypes = [i32, i32, i32, i32]
    lib.sv_verify_greedy_workspace.restype = sz
    lib.sv_verify_greedy.argtypes = [SvRows, i32, i32, i32, P, P, P, P, P, P, sz, P]
    lib.sv_verify_greedy.restype = C.c_int
    lib.sv_verify_greedy_top2_workspace.argtypes = [i32, i32, i32, i32]
    lib.sv_verify_greedy_top2_workspace.restype = sz
    lib.sv_verify_greedy_top2.argtypes = [SvRows, i32, i32, i32, P, P, P, P, P, P, P, sz, P]
    lib.sv_verify_greedy_top2.restype = C.c_int
    lib.sv_infer_modality_workspace.argtypes = [i32, i32]
    lib.sv_infer_modality_workspace.restype = sz
    lib.sv_infer_modality.argtypes = [SvRows, i32, P, i32, P, P, P, P, P, P, sz, P]
    lib.sv_infer_modality.restype = C.c_int
    lib.sv_verify_sample_workspace.argtypes = [i32, i32, i32, i32]
    lib.sv_verify_sample_workspace.restype = sz
    lib.sv_verify_sample.argtypes = [SvRows, SvRows, P, P, i32, i32, P, P, P, P, P, P, P, P, P, P, sz, P]
    lib.sv_d2t_plan_bytes.argtypes = [i32, i32]
    lib.sv_d2t_plan_bytes.restype = sz
    lib.sv_d2t_plan_build.argtypes = [P, i32, i32, P, sz, P]
    lib.sv_d2t_plan_build.restype = C.c_int
    lib.sv_verify_sample.restype = C.c_int
    lib.sv_cfg_merge_sample_workspace.argtypes = [i32, i32, i32, i32]
    lib.sv_cfg_merge_sample_workspace.restype = sz
    lib.sv_cfg_merge_sample.argtypes = [SvRows, SvRows, P, P, i32, f32, SvRows, i32, i32, P, P, P, P, P, P,
                                        P, P, sz, P]
    lib.sv_cfg_merge_sample.restype = C.c_int
    lib.sv_pool_append.argtypes = [P, P, i32, P, i32, i32, P, P]
    lib.sv_pool_lookup.argtypes = [P, P, i32, P, i32, i32, i32, P, P, P]
    lib.sv_suffix_append.argtypes = [P, i32, i32, P, P, i32, P]
    lib.sv_accept_scan.argtypes = [P, P, P, i32, i32, P, P, P]
    lib.sv_accept_scan.restype = C.c_int
    i64, f64 = C.c_int64, C.c_double
    lib.sv_step_tables.argtypes = [P, P, i32, i32, P, i32, P, P, i32, P, i32, P, P, P, P, P, i32, P, P, P]
    lib.sv_rope_cache.argtypes = [SvHeads, SvHeads, SvHeads, P, P, P, i32, i32, f32, SvHeads, SvKvCache, P]
    lib.sv_rope_freqs.argtypes = [i32, f64, i32, f64, f64, f64, f64, P]
    lib.sv_tree_attention_workspace.argtypes = [i32, i32, i32, i32, i32, i32, i64]
    lib.sv_tree_attention_workspace.restype = sz
    lib.sv_tree_attention.argtypes = [SvHeads, SvKvCache, P, i32, P, P, i32, i32, P, i32, f32, SvHeads, P, P, P, sz, P]
    lib.sv_selftest_tree_attention_stop.argtypes = lib.sv_tree_attention.argtypes[:-1] + [i32, P]
    lib.sv_cache_commit.argtypes = [SvKvCache, P, i32, P, P, P, i32, P, P, P, i32, P, P, P, P, P, P]
    lib.sv_selftest_wait_timeout.argtypes = [P, P, C.c_int64, P]
    lib.sv_selftest_wait_timeout.restype = C.c_int
    _lib = lib
    return lib


def _check(rc: int):
    if rc != 0:
        raise SpecVerifyError(rc, load().sv_status_string(rc).decode())


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def rows_of(t, width: int | None = None) -> SvRows:
    """Describe a 2-D CUDA tensor of logits (rows may be strided)."""
    import torch

    if t is None:
        return SvRows(None, SV_F32, int(width or 1), 0)
    if not t.is_cuda or t.dim() != 2:
        raise ValueError("logits must be a 2-D CUDA tensor")
    if t.dtype == torch.bfloat16:
        code = SV_BF16
    elif t.dtype == torch.float32:
        code = SV_F32
    else:
        raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")
    if t.shape[0] > 1 and t.stride(1) != 1:
        raise ValueError("entries of a logit row must be contiguous")
    stride = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    return SvRows(t.data_ptr(), code, int(width if width is not None else t.shape[1]), int(stride))


def _empty(shape, dtype, device, stream=None):
    """An output.  It is made on the stream that writes it: the current one's memory may still be read by work ahead of
    the call.  The caller's stream is noted, as that is where it will be read."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _workspace(nbytes, device, workspace, stream=None):
    """The given workspace, or one made on the stream that uses it, which gets its memory back."""
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace needs {nbytes} bytes")
        return workspace
    if stream is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _nbytes(t):
    return t.numel() * t.element_size()


def verify_greedy_workspace(R: int, k: int, branches: int, V: int) -> int:
    return int(load().sv_verify_greedy_workspace(R, k, branches, V))


def verify_greedy(target, R: int, k: int, branches: int, draft, out: dict | None = None, workspace=None,
                  stream=None) -> dict:
    """Greedy verification.  target: [R*rows_per_request, V] bf16/f32 CUDA
    tensor; draft: int32 [R, branches, k].  Returns accept_len [R], tokens
    [R, k+1], branch [R], status [R] (int32 CUDA tensors)."""
    import torch

    lib = load()
    dev = target.device
    if out is None:
        out = dict(accept_len=_empty(R, torch.int32, dev, stream), tokens=_empty((R, k + 1), torch.int32, dev, stream),
                   branch=_empty(R, torch.int32, dev, stream), status=_empty(R, torch.int32, dev, stream))
    ws = _workspace(lib.sv_verify_greedy_workspace(R, k, branches, target.shape[1]), dev, workspace, stream)
    _check(lib.sv_verify_greedy(rows_of(target), R, k, branches, _ptr(draft), _ptr(out["accept_len"]),
                                _ptr(out["tokens"]), _ptr(out.get("branch")), _ptr(out.get("status")), _ptr(ws),
                                _nbytes(ws), _stream(stream)))
    return out


def verify_greedy_top2_workspace(R: int, k: int, branches: int, V: int) -> int:
    return int(load().sv_verify_greedy_top2_workspace(R, k, branches, V))


def verify_greedy_top2(target, R: int, k: int, branches: int, draft, out: dict | None = None, workspace=None,
                       stream=None) -> dict:
    """verify_greedy plus top2 [rows, 2]: per row the argmax and the runner-up id
    (logit descending, then id ascending; -1 when V == 1), from the same pass."""
    import torch

    lib = load()
    dev = target.device
    rows = target.shape[0] if R == 0 else R * (1 + branches * k)
    if out is None:
        out = dict(accept_len=_empty(R, torch.int32, dev, stream), tokens=_empty((R, k + 1), torch.int32, dev, stream),
                   branch=_empty(R, torch.int32, dev, stream), status=_empty(R, torch.int32, dev, stream),
                   top2=_empty((rows, 2), torch.int32, dev, stream))
    ws = _workspace(lib.sv_verify_greedy_top2_workspace(R, k, branches, target.shape[1]), dev, workspace, stream)
    _check(lib.sv_verify_greedy_top2(rows_of(target), R, k, branches, _ptr(draft), _ptr(out["accept_len"]),
                                     _ptr(out["tokens"]), _ptr(out.get("branch")), _ptr(out.get("status")),
                                     _ptr(out["top2"]), _ptr(ws), _nbytes(ws), _stream(stream)))
    return out


def infer_modality(logits, part_start, out: dict | None = None, workspace=None, stream=None) -> dict:
    """Per row of full-vocabulary logits [N, V]: amax, the partition holding it (part, -1 for
    none) and its id range (mask_lo, mask_hi), with status bits.  part_start: host ints,
    ascending, P + 1 of them."""
    import numpy as np
    import torch

    lib = load()
    dev = logits.device
    N = logits.shape[0]
    ps = np.ascontiguousarray(np.asarray(part_start, dtype=np.int32))
    if out is None:
        out = {key: _empty(N, torch.int32, dev, stream) for key in ("amax", "part", "mask_lo", "mask_hi", "status")}
    ws = _workspace(lib.sv_infer_modality_workspace(N, logits.shape[1]), dev, workspace, stream)
    _check(lib.sv_infer_modality(rows_of(logits), N, ps.ctypes.data, ps.size - 1, _ptr(out.get("amax")),
                                 _ptr(out["part"]), _ptr(out.get("mask_lo")), _ptr(out.get("mask_hi")),
                                 _ptr(out.get("status")), _ptr(ws), _nbytes(ws), _stream(stream)))
    return out


def verify_sample_workspace(R: int, k: int, V: int, Vd: int) -> int:
    return int(load().sv_verify_sample_workspace(R, k, V, Vd))


def d2t_plan(d2t, V: int, stream=None):
    """Build the device-side plan of a d2t map once (a uint8 CUDA tensor) for
    verify_sample(..., plan=...)."""
    import torch

    lib = load()
    Vd = d2t.numel()
    nbytes = int(lib.sv_d2t_plan_bytes(V, Vd))
    plan = _empty(nbytes, torch.uint8, d2t.device, stream)
    _check(lib.sv_d2t_plan_build(_ptr(d2t), Vd, V, _ptr(plan), nbytes, _stream(stream)))
    return plan


def verify_sample(target, draft_logits, d2t, R: int, k: int, draft, seeds, temperature, out: dict | None = None,
                  workspace=None, stream=None, stats: bool = True, plan=None) -> dict:
    """Speculative sampling.  target [R*(k+1), V]; draft_logits [R*k, Vd];
    d2t int32 [Vd] or None; draft int32 [R, k]; seeds uint64 bits in an int64
    tensor [R]; temperature float32 [R]; plan: d2t_plan(d2t, V) or None.
    Returns accept_len, tokens, status and, with stats=True, tv / p_draft /
    q_draft [R, k]."""
    import torch

    lib = load()
    dev = target.device
    V = target.shape[1]
    if draft_logits is not None:
        Vd = draft_logits.shape[1]
    else:
        Vd = V if d2t is None else d2t.numel()
    if out is None:
        out = dict(accept_len=_empty(R, torch.int32, dev, stream), tokens=_empty((R, k + 1), torch.int32, dev, stream),
                   status=_empty(R, torch.int32, dev, stream))
        if stats:
            for name in ("tv", "p_draft", "q_draft"):
                out[name] = _empty((R, k), torch.float32, dev, stream)
    ws = _workspace(lib.sv_verify_sample_workspace(R, k, V, Vd), dev, workspace, stream)
    _check(lib.sv_verify_sample(rows_of(target), rows_of(draft_logits, Vd), _ptr(d2t), _ptr(plan), R, k, _ptr(draft),
                                _ptr(seeds), _ptr(temperature), _ptr(out["accept_len"]), _ptr(out["tokens"]),
                                _ptr(out.get("tv")), _ptr(out.get("p_draft")), _ptr(out.get("q_draft")),
                                _ptr(out.get("status")), _ptr(ws), _nbytes(ws), _stream(stream)))
    return out


def cfg_merge_sample_workspace(R: int, k: int, S: int, W: int) -> int:
    return int(load().sv_cfg_merge_sample_workspace(R, k, S, W))


def cfg_merge_sample(cond, uncond, cb_id_base, cb_data_offset, S: int, W: int, w: float, draft_logits, R: int,
                     k: int, draft, seeds, temperature, out: dict | None = None, workspace=None, stream=None,
                     stats: bool = True) -> dict:
    """CFG merge per codebook, then verification.  cond/uncond [R*(k+1)*S, row]
    with codebook s at element cb_data_offset[s] (W entries); cb_id_base and
    cb_data_offset are host int sequences of length S; draft_logits
    [R*k*S, W] or None (greedy); draft int32 [R, k, S] absolute ids."""
    import torch

    lib = load()
    dev = cond.device
    if out is None:
        out = dict(accept_len=_empty(R, torch.int32, dev, stream),
                   tokens=_empty((R, k + 1, S), torch.int32, dev, stream),
                   status=_empty(R, torch.int32, dev, stream))
        if stats:
            out["tv"] = _empty((R, k, S), torch.float32, dev, stream)
    base = (C.c_int32 * S)(*[int(b) for b in cb_id_base])
    off = None if cb_data_offset is None else (C.c_int32 * S)(*[int(o) for o in cb_data_offset])
    ws = _workspace(lib.sv_cfg_merge_sample_workspace(R, k, S, W), dev, workspace, stream)
    _check(lib.sv_cfg_merge_sample(rows_of(cond, W), rows_of(uncond, W), C.cast(base, C.c_void_p),
                                   None if off is None else C.cast(off, C.c_void_p), S, float(w),
                                   rows_of(draft_logits, W), R, k, _ptr(draft), _ptr(seeds), _ptr(temperature),
                                   _ptr(out["accept_len"]), _ptr(out["tokens"]), _ptr(out.get("tv")),
                                   _ptr(out.get("status")), _ptr(ws), _nbytes(ws), _stream(stream)))
    return out


def pool_append(pool, pool_len, drafts, status=None, stream=None):
    """Insert drafts int32 [R, k] (a negative id ends a draft early) into the pools
    int32 [R, Lp] whose used lengths are pool_len int32 [R]; both are updated in
    place.  status int32 [R] (optional) gets SV_ST_POOL_FULL where a draft did not fit."""
    lib = load()
    R, Lp = pool.shape
    k = drafts.shape[1]
    _check(lib.sv_pool_append(_ptr(pool), _ptr(pool_len), Lp, _ptr(drafts), k, R, _ptr(status), _stream(stream)))
    return status


def pool_lookup(pool, pool_len, suffix, gamma: int, out: dict | None = None, stream=None) -> dict:
    """Longest n-gram of the pools int32 [R, Lp] (used lengths pool_len int32 [R])
    matching the emitted suffix int32 [R, N] (-1 padded on the left); returns
    match_len int32 [R] and the continuation cont int32 [R, gamma] (-1 padded)."""
    import torch

    lib = load()
    R, Lp = pool.shape
    N = suffix.shape[1]
    dev = pool.device
    if out is None:
        out = dict(match_len=_empty(R, torch.int32, dev, stream), cont=_empty((R, gamma), torch.int32, dev, stream))
    _check(lib.sv_pool_lookup(_ptr(pool), _ptr(pool_len), Lp, _ptr(suffix), N, R, gamma, _ptr(out["match_len"]),
                              _ptr(out["cont"]), _stream(stream)))
    return out


def suffix_append(suffix, tokens, accept_len, stream=None):
    """Shift a verify step's committed tokens (tokens int32 [R, k + 1], entries 0..n with
    n = accept_len[r]) into the emitted suffix int32 [R, N], in place."""
    lib = load()
    R, N = suffix.shape
    k = tokens.shape[1] - 1
    _check(lib.sv_suffix_append(_ptr(suffix), N, R, _ptr(tokens), _ptr(accept_len), k, _stream(stream)))
    return suffix


def accept_scan(accept, draft, fix, out: dict | None = None, stream=None) -> dict:
    """accept uint8 [R, k]; draft int32 [R, k]; fix int32 [R, k+1]."""
    import torch

    lib = load()
    R, k = accept.shape
    dev = accept.device
    if out is None:
        out = dict(accept_len=_empty(R, torch.int32, dev, stream), tokens=_empty((R, k + 1), torch.int32, dev, stream))
    _check(lib.sv_accept_scan(_ptr(accept), _ptr(draft), _ptr(fix), R, k, _ptr(out["accept_len"]),
                              _ptr(out["tokens"]), _stream(stream)))
    return out


def _half_type(t) -> int:
    if t.dtype is torch.bfloat16:
        return SV_BF16
    if t.dtype is torch.float16:
        return SV_F16
    raise TypeError(f"heads and caches must be bfloat16 or float16, got {t.dtype}")


def heads_of(t) -> SvHeads:
    """Describe a CUDA tensor of heads [tokens, heads, head_dim] (tokens and heads may be strided)."""
    load()
    if not t.is_cuda or t.dim() != 3:
        raise ValueError("heads must be a 3-D CUDA tensor [tokens, heads, head_dim]")
    T, H, D = t.shape
    st, sh, sd = t.stride()
    if sd != 1 and D > 1:
        raise ValueError("entries of a head must be contiguous")
    return SvHeads(t.data_ptr(), _half_type(t), T, H, D, st, sh)


def cache_of(k, v) -> SvKvCache:
    """Describe a paged cache: K and V tensors [num_blocks, block_size, kv_heads, head_dim], or with the layers in
    front, of one dtype and the same strides (any order of the axes but the last)."""
    load()
    shape, strides = k.shape, k.stride()
    n = len(shape)
    if not k.is_cuda or not v.is_cuda or n not in (4, 5) or shape != v.shape:
        raise ValueError("caches must be 4-D or 5-D CUDA tensors of one shape")
    if k.dtype is not v.dtype:
        raise TypeError("K and V caches must have one dtype")
    if strides != v.stride():
        raise ValueError("K and V caches must have the same strides")
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError("entries of a head must be contiguous")
    layers, layer_stride = (1, 0) if n == 4 else (shape[0], strides[0])
    nb, bs, H, D = shape[-4:]
    sb, st, sh, _ = strides[-4:]
    return SvKvCache(k.data_ptr(), v.data_ptr(), _half_type(k), nb, bs, H, D, layers, sb, st, sh, layer_stride)


def _ints(t, name, n=-1) -> int:
    """The address of an int32 CUDA tensor that is passed as it lies."""
    if t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    if n >= 0 and t.numel() != n:
        raise ValueError(f"{name} must have {n} entries, got {t.numel()}")
    return t.data_ptr()


def _check_out(out, **want):
    """Tensors that a caller gave for outputs must have room for what the kernels write: name=(dtype, entries)."""
    for name, (dtype, n) in want.items():
        t = out.get(name)
        if t is not None and (t.dtype is not dtype or not t.is_cuda or not t.is_contiguous() or t.numel() < n):
            raise ValueError(f"out[{name!r}] must be a contiguous {dtype} CUDA tensor with room for {n} entries")


def _at(t):
    return None if t is None else t.data_ptr()


def _raw_stream(stream, t) -> int:
    """The given stream's handle, or the current one's (without building a stream object for it).  The library launches
    on the current device, which has to be the one of the tensors."""
    device = torch._C._cuda_getDevice()
    if t.get_device() != device:
        raise ValueError(f"a tensor is on {t.device}, but cuda:{device} is the current device")
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _new_ints(like, stream, *sizes):
    """Int32 tensors of these sizes in one allocation and one split: allocating each costs more than the launch that
    fills them."""
    return torch.unsafe_split_with_sizes(_empty(sum(sizes), torch.int32, like.device, stream), sizes)


def step_tables(seq_len, new_len, block_table, free_blocks, free_count, block_size: int, T: int, parent=None,
                mask_words: int = 0, out: dict | None = None, stream=None) -> dict:
    """Lay a step's tokens out in the paged cache.  seq_len, new_len int32 [R]; block_table int32
    [R, max_blocks], whose new entries are written in place; free_blocks int32 [num_blocks] with free_count
    int32 [1] of them free; T the capacity of the packed arrays; parent int32 [T] or None (a chain).  Returns
    cu_tokens [R + 1], kv_len [R], slot int64 [T], position [T], free_count [1], status [R] and, with parents,
    mask int32 [T, mask_words] (ancestor bits)."""
    lib = load()
    R = seq_len.numel()
    if block_table.dim() != 2 or block_table.shape[0] != R:
        raise ValueError("block_table must be [R, max_blocks]")
    a_seq, a_table = _ints(seq_len, "seq_len"), _ints(block_table, "block_table")
    if out is None:
        # the 64-bit slots lie first, as pairs of 32-bit entries
        slot, cu, kv, position, count, status, mask = _new_ints(
            seq_len, stream, 2 * T, R + 1, R, T, 1, R, T * mask_words if parent is not None else 0)
        out = dict(cu_tokens=cu, kv_len=kv, slot=slot.view(torch.int64), position=position, free_count=count,
                   status=status)
        if parent is not None:
            out["mask"] = mask.view(T, mask_words)
    else:
        i32 = torch.int32
        _check_out(out, cu_tokens=(i32, R + 1), kv_len=(i32, R), slot=(torch.int64, T), position=(i32, T),
                   free_count=(i32, 1), status=(i32, R))
        if parent is not None:
            _check_out(out, mask=(i32, T * mask_words))
            if out["mask"].dim() == 2 and out["mask"].shape[1] != mask_words:
                raise ValueError(f"out['mask'] must have rows of {mask_words} words")
    mask = out.get("mask") if parent is not None else None
    if R == 0:  # nothing to lay out
        with torch.cuda.stream(stream):
            out["cu_tokens"].zero_()
            out["free_count"].copy_(free_count)
            for name in ("slot", "position"):
                out[name].fill_(-1)
            if mask is not None:
                mask.zero_()
        return out
    rc = lib.sv_step_tables(a_seq, _ints(new_len, "new_len", R), R, block_size, a_table, block_table.shape[1],
                            _ints(free_blocks, "free_blocks"), _ints(free_count, "free_count", 1),
                            free_blocks.numel(), None if parent is None else _ints(parent, "parent", T), T,
                            out["cu_tokens"].data_ptr(), out["kv_len"].data_ptr(), out["slot"].data_ptr(),
                            out["position"].data_ptr(), _at(mask), mask_words if mask is not None else 0,
                            out["free_count"].data_ptr(), _at(out.get("status")), _raw_stream(stream, seq_len))
    if rc:
        _check(rc)
    return out


def rope_freqs(rot_dim: int, base: float = 10000.0, scaling: int = ROPE_PLAIN, factor: float = 1.0,
               trained: float = 0.0, low: float = 0.0, high: float = 0.0, device="cuda"):
    """Frequencies for rope_cache: an int64 tensor [rot_dim / 2] of 64-bit turn fractions (see sv_rope_freqs for
    the scalings).  rope_cache takes them on the GPU."""
    lib = load()
    host = torch.zeros(max(rot_dim, 0) // 2, dtype=torch.int64)
    _check(lib.sv_rope_freqs(rot_dim, base, scaling, factor, trained, low, high, _ptr(host)))
    return host.to(device)


def rope_cache(q, k, v, position, slot, freqs, k_cache, v_cache, interleaved: bool = False, mscale: float = 1.0,
               q_out=None, stream=None):
    """Rotate q [T, heads, D] and k [T, kv_heads, D] at position int32 [T] and write k and v into the paged cache
    at slot int64 [T] (-1: not cached).  freqs: rope_freqs(rot_dim).  Returns the rotated q (q_out may be q)."""
    lib = load()
    T = q.shape[0]
    if q_out is None:
        q_out = _empty(q.shape, q.dtype, q.device, stream)
    if slot.dtype is not torch.int64 or not slot.is_cuda or not slot.is_contiguous() or slot.numel() != T:
        raise ValueError("slot must be a contiguous int64 CUDA tensor with an entry for each token")
    if freqs.dtype not in (torch.int64, torch.uint64) or not freqs.is_cuda or not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous int64 CUDA tensor from rope_freqs")
    rc = lib.sv_rope_cache(heads_of(q), heads_of(k), heads_of(v), _ints(position, "position", T), slot.data_ptr(),
                           freqs.data_ptr(), 2 * freqs.numel(), 1 if interleaved else 0, mscale, heads_of(q_out),
                           cache_of(k_cache, v_cache), _raw_stream(stream, q))
    if rc:
        _check(rc)
    return q_out


def tree_attention_workspace(R: int, T: int, max_tokens: int, heads: int, kv_heads: int, head_dim: int,
                             max_kv: int) -> int:
    return int(load().sv_tree_attention_workspace(R, T, max_tokens, heads, kv_heads, head_dim, max_kv))


def tree_attention(q, k_cache, v_cache, block_table, kv_len, cu_tokens, max_tokens: int, mask=None,
                   scale: float | None = None, with_lse: bool = False, out: dict | None = None, workspace=None,
                   stream=None, with_status: bool = False) -> dict:
    """Attention of the packed step tokens q [T, heads, D] over the paged cache.  block_table int32
    [R, max_blocks]; kv_len int32 [R]; cu_tokens int32 [R + 1]; max_tokens bounds a request's tokens; mask int32
    [T, words] (which of its request's step tokens a token sees) or None (a chain); scale defaults to
    D ** -0.5.  Returns out [T, heads, D] and, with_lse, lse float32 [T, heads]; with_status, status int32 [R],
    which is ST_TIMEOUT for every request when a wait on the device gave up.  out and lse are then NaN.  Rows of
    tokens that do not attend (behind cu_tokens[R], or a request's behind max_tokens) are not written."""
    lib = load()
    T, heads, D = q.shape
    R, max_blocks = block_table.shape
    if out is None:
        out = dict(out=_empty(q.shape, q.dtype, q.device, stream))
        if with_lse:
            out["lse"] = _empty((T, heads), torch.float32, q.device, stream)
        if with_status:
            out["status"] = _empty(R, torch.int32, q.device, stream)
    else:
        _check_out(out, lse=(torch.float32, T * heads), status=(torch.int32, R))
    if mask is not None and (mask.dim() != 2 or mask.shape[0] != T):
        raise ValueError("mask must be [T, words]")
    cache = cache_of(k_cache, v_cache)
    if workspace is None:
        workspace = _workspace(lib.sv_tree_attention_workspace(R, T, max_tokens, heads, cache.kv_heads, D,
                                                               max_blocks * cache.block_size), q.device, None, stream)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    rc = lib.sv_tree_attention(heads_of(q), cache, _ints(block_table, "block_table"), max_blocks,
                               _ints(kv_len, "kv_len", R), _ints(cu_tokens, "cu_tokens", R + 1), R, max_tokens,
                               None if mask is None else _ints(mask, "mask"), 0 if mask is None else mask.shape[1],
                               D ** -0.5 if scale is None else scale, heads_of(out["out"]), _at(out.get("lse")),
                               _at(out.get("status")), workspace.data_ptr(), _nbytes(workspace), _raw_stream(stream, q))
    if rc:
        _check(rc)
    return out


def cache_commit(k_cache, v_cache, block_table, seq_len, kv_len, cu_tokens, accept_len, k: int, free_blocks,
                 free_count, branch=None, path=None, out: dict | None = None, stream=None) -> dict:
    """Keep the accepted path of a verified tree: the accepted drafts' keys and values move behind the root in every
    layer of the caches ([layers, ] num_blocks, block_size, kv_heads, head_dim), and the blocks without a kept token
    are pushed on free_blocks.  accept_len int32 [R] and branch int32 [R] as verify_greedy returns them, or path
    int32 [R, k] of the accepted tokens' numbers.  Returns seq_len [R], free_count [1] and status [R]."""
    lib = load()
    R = seq_len.numel()
    if block_table.dim() != 2 or block_table.shape[0] != R:
        raise ValueError("block_table must be [R, max_blocks]")
    a_seq = _ints(seq_len, "seq_len")
    if out is None:
        out = dict(zip(("seq_len", "free_count", "status"), _new_ints(seq_len, stream, R, 1, R)))
    else:
        _check_out(out, seq_len=(torch.int32, R), free_count=(torch.int32, 1), status=(torch.int32, R))
    if R == 0:
        with torch.cuda.stream(stream):
            out["free_count"].copy_(free_count)
        return out
    rc = lib.sv_cache_commit(cache_of(k_cache, v_cache), _ints(block_table, "block_table"), block_table.shape[1], a_seq,
                             _ints(kv_len, "kv_len", R), _ints(cu_tokens, "cu_tokens", R + 1), R,
                             _ints(accept_len, "accept_len", R), None if branch is None else _ints(branch, "branch", R),
                             None if path is None else _ints(path, "path", R * k), k,
                             _ints(free_blocks, "free_blocks", k_cache.shape[-4]), _ints(free_count, "free_count", 1),
                             out["seq_len"].data_ptr(), out["free_count"].data_ptr(), _at(out.get("status")),
                             _raw_stream(stream, seq_len))
    if rc:
        _check(rc)
    return out


def selftest_wait_timeout(limit_cycles: int, stream=None):
    """Make one bounded barrier wait of the library run out on purpose (sv_selftest_wait_timeout);
    returns the int32 [2] device status: [0] the timeout bit, [1] whether the real copy landed."""
    import torch

    src = torch.arange(4, dtype=torch.int32, device="cuda") + 0x5A5A0000
    status = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    _check(load().sv_selftest_wait_timeout(_ptr(src), _ptr(status), limit_cycles, _stream(stream)))
    return status
