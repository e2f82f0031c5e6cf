"""GB300-native DiffusionGemma per-row sampler statistics.

A thin ctypes binding of ``libdrs.so`` (declared in ``include/drs.h``). Every
function here only marshals arguments: pointers of torch tensors, sizes, the
current CUDA stream. All of the arithmetic runs in the library's CUDA kernels;
there is no CPU fallback. Importing the package works without a GPU; calling
into the library needs the built ``libdrs.so`` and a CUDA device, and raises
otherwise.

Entry points (same names as the C ABI):
  drs_row_stats, drs_row_stats_workspace_bytes, drs_row_stats_noalloc,
  drs_row_stats_topk, drs_row_stats_topk_workspace_bytes, drs_topk_logprobs,
  drs_topk_workspace_bytes, drs_philox_gumbel, drs_scaled_logits,
  drs_stash_converged_logprobs, drs_stash_workspace_bytes,
  drs_verify_drafts, drs_map_slots, drs_embed_tokens, drs_embed_tokens_grad,
  drs_embed_tokens_grad_workspace_bytes, drs_token_logprobs,
  drs_token_logprobs_grad, drs_dropout, drs_dropout_grad,
  drs_status_string, drs_get_device_error.
Convenience wrappers that allocate outputs: row_stats, row_stats_topk,
topk_logprobs, philox_gumbel, stash_converged_logprobs, verify_drafts,
map_slots, embed_tokens, embed_tokens_grad, token_logprobs,
token_logprobs_grad, dropout, dropout_grad.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

from . import _build

DRS_OK = 0
DRS_ERR_INVALID_ARG = -1
DRS_ERR_UNSUPPORTED = -2
DRS_ERR_CUDA = -3
DRS_ERR_DEVICE_TIMEOUT = -4

DRS_PROBS_NONE, DRS_PROBS_BF16, DRS_PROBS_FP16 = 0, 1, 2
DRS_DTYPE_FP32, DRS_DTYPE_BF16, DRS_DTYPE_FP16 = 0, 1, 2
DRS_MAX_VOCAB = 2097152
DRS_MAX_REQUESTS = 1048576
DRS_MAX_TOKENS = 268435456
DRS_MAX_WIDTH = 1048576
DRS_MAX_ALTERNATIVES = 64
DRS_MAX_SCORE_ROWS = 134217727

EXPORTED = ("drs_row_stats", "drs_row_stats_workspace_bytes", "drs_row_stats_noalloc",
            "drs_row_stats_topk", "drs_row_stats_topk_workspace_bytes", "drs_topk_logprobs",
            "drs_topk_workspace_bytes", "drs_philox_gumbel", "drs_scaled_logits",
            "drs_status_string", "drs_get_device_error", "drs_test_inject_fault",
            "drs_kernel_timing", "drs_kernel_times", "drs_row_stats_seeds",
            "drs_row_stats_seeds_workspace_bytes", "drs_stash_converged_logprobs",
            "drs_stash_workspace_bytes", "drs_test_two_pass",
            "drs_row_split_plan", "drs_verify_drafts", "drs_map_slots", "drs_embed_tokens",
            "drs_embed_tokens_grad", "drs_embed_tokens_grad_workspace_bytes", "drs_token_logprobs",
            "drs_token_logprobs_grad", "drs_dropout", "drs_dropout_grad")


class DrsError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libdrs.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB_PATH
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(f"libdrs.so is not built ({path}); run "
                               "vocab_row_sampling_gb300._build.build()")
        _build.build()
    lib = ctypes.CDLL(path)
    i64, u64, i32, vp, sz = (ctypes.c_int64, ctypes.c_uint64, ctypes.c_int32,
                             ctypes.c_void_p, ctypes.c_size_t)
    lib.drs_row_stats_workspace_bytes.argtypes = [i64, i64]
    lib.drs_row_stats_workspace_bytes.restype = sz
    lib.drs_row_stats.argtypes = [vp, i64, i64, i64, vp, i64, u64, i64, vp, vp, vp,
                                  ctypes.c_int, vp, i64, vp, sz, vp]
    lib.drs_row_stats.restype = ctypes.c_int
    lib.drs_row_stats_noalloc.argtypes = [vp, i64, i64, i64, vp, i64, u64, i64, vp, vp, vp,
                                          ctypes.c_int, vp, i64, vp]
    lib.drs_row_stats_noalloc.restype = ctypes.c_int
    lib.drs_row_stats_topk_workspace_bytes.argtypes = [i64, i64, i32]
    lib.drs_row_stats_topk_workspace_bytes.restype = sz
    lib.drs_row_stats_topk.argtypes = [vp, i64, i64, i64, vp, i64, u64, i64, vp, vp, vp,
                                       ctypes.c_int, vp, i64, vp, i32, vp, vp, vp, sz, vp]
    lib.drs_row_stats_topk.restype = ctypes.c_int
    lib.drs_topk_workspace_bytes.argtypes = [i64, i64, i32]
    lib.drs_topk_workspace_bytes.restype = sz
    lib.drs_topk_logprobs.argtypes = [vp, i64, i64, i64, vp, i64, vp, i32, vp, vp, vp, sz, vp]
    lib.drs_topk_logprobs.restype = ctypes.c_int
    lib.drs_stash_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.drs_stash_workspace_bytes.restype = sz
    lib.drs_stash_converged_logprobs.argtypes = [vp, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp,
                                                 i32, vp, vp, i64, i64, i32, vp, vp, vp,
                                                 ctypes.c_int, vp, sz, vp]
    lib.drs_stash_converged_logprobs.restype = ctypes.c_int
    lib.drs_philox_gumbel.argtypes = [u64, i64, i64, i64, vp, vp, vp]
    lib.drs_philox_gumbel.restype = ctypes.c_int
    lib.drs_scaled_logits.argtypes = [vp, i64, ctypes.c_float, vp, vp]
    lib.drs_scaled_logits.restype = ctypes.c_int
    lib.drs_status_string.argtypes = [ctypes.c_int]
    lib.drs_status_string.restype = ctypes.c_char_p
    lib.drs_test_inject_fault.argtypes = [ctypes.c_int]
    lib.drs_test_inject_fault.restype = None
    lib.drs_test_two_pass.argtypes = [ctypes.c_int]
    lib.drs_test_two_pass.restype = None
    lib.drs_row_split_plan.argtypes = [i64, i64, i32, i32, ctypes.c_int, i32, vp, vp, vp, vp]
    lib.drs_row_split_plan.restype = ctypes.c_int
    lib.drs_get_device_error.argtypes = [vp]
    lib.drs_get_device_error.restype = ctypes.c_int
    lib.drs_row_stats_seeds_workspace_bytes.argtypes = [i64, i64, i32]
    lib.drs_row_stats_seeds_workspace_bytes.restype = sz
    lib.drs_row_stats_seeds.argtypes = [vp, i64, i64, i64, vp, i64, vp, i32, i64, vp, vp, vp,
                                        ctypes.c_int, vp, i64, vp, sz, vp]
    lib.drs_row_stats_seeds.restype = ctypes.c_int
    lib.drs_kernel_timing.argtypes = [ctypes.c_int]
    lib.drs_kernel_timing.restype = ctypes.c_int
    lib.drs_kernel_times.argtypes = [vp, i32, vp]
    lib.drs_kernel_times.restype = ctypes.c_int
    lib.drs_verify_drafts.argtypes = [vp, ctypes.c_int, i64, i64, vp, ctypes.c_int, i64, i64, i64,
                                      vp, vp, i64, i32, vp, vp, vp, vp, vp]
    lib.drs_verify_drafts.restype = ctypes.c_int
    lib.drs_map_slots.argtypes = [vp, vp, vp, i64, i32, vp, i64, i32, vp, i64, vp, i64, vp, vp, vp,
                                  vp, vp, vp, vp, vp]
    lib.drs_map_slots.restype = ctypes.c_int
    lib.drs_embed_tokens.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, i32, i64, ctypes.c_float,
                                     vp, i64, vp]
    lib.drs_embed_tokens.restype = ctypes.c_int
    lib.drs_embed_tokens_grad_workspace_bytes.argtypes = [i64, i64, i64]
    lib.drs_embed_tokens_grad_workspace_bytes.restype = sz
    lib.drs_embed_tokens_grad.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, i32, ctypes.c_float,
                                          ctypes.c_int, vp, ctypes.c_int, i64, i64, vp, sz, vp]
    lib.drs_embed_tokens_grad.restype = ctypes.c_int
    lib.drs_token_logprobs.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, i32, vp, i64, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.drs_token_logprobs.restype = ctypes.c_int
    lib.drs_token_logprobs_grad.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, i32, vp, i64, vp, vp, vp, vp, vp,
                                            ctypes.c_int, i64, vp]
    lib.drs_token_logprobs_grad.restype = ctypes.c_int
    lib.drs_dropout.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, i64, ctypes.c_float, u64, vp, i64, vp,
                                ctypes.c_int, i64, vp]
    lib.drs_dropout.restype = ctypes.c_int
    lib.drs_dropout_grad.argtypes = [vp, ctypes.c_int, i64, i64, i64, ctypes.c_float, u64, vp, i64, vp, ctypes.c_int,
                                     i64, vp]
    lib.drs_dropout_grad.restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().drs_status_string(status).decode()


drs_status_string = status_string


def _check(status: int, what: str):
    if status != DRS_OK:
        raise DrsError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _row_stride(logits) -> int:
    assert logits.dim() == 2 and logits.stride(1) == 1, "logits: 2-D, unit column stride"
    return logits.stride(0) if logits.shape[0] > 1 else max(logits.shape[1], logits.stride(0))


# ------------------------------------------------------------- raw entry points

def drs_row_stats_workspace_bytes(rows: int, vocab: int) -> int:
    return int(load().drs_row_stats_workspace_bytes(rows, vocab))


def drs_row_stats(logits, temps, canvas_len, seed, argmax, sample, entropy,
                  probs_dtype=DRS_PROBS_NONE, probs=None, workspace=None, stream=None,
                  row0=0):
    """Launch drs_row_stats on torch CUDA tensors (outputs preallocated)."""
    rows, vocab = logits.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    pstride = 0 if probs is None else probs.stride(0)
    st = load().drs_row_stats(_ptr(logits), rows, vocab, _row_stride(logits), _ptr(temps),
                              canvas_len, seed & (2**64 - 1), row0, _ptr(argmax), _ptr(sample),
                              _ptr(entropy), probs_dtype, _ptr(probs), pstride,
                              _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "drs_row_stats")


def drs_row_stats_noalloc(logits, temps, canvas_len, seed, argmax, sample, entropy,
                          probs_dtype=DRS_PROBS_NONE, probs=None, stream=None, row0=0):
    """drs_row_stats with the library's fixed device workspace: for callers
    that cannot allocate device memory (see include/drs.h). Calls that can
    overlap on the GPU share that workspace and race."""
    rows, vocab = logits.shape
    pstride = 0 if probs is None else probs.stride(0)
    st = load().drs_row_stats_noalloc(_ptr(logits), rows, vocab, _row_stride(logits),
                                      _ptr(temps), canvas_len, seed & (2**64 - 1), row0,
                                      _ptr(argmax), _ptr(sample), _ptr(entropy), probs_dtype,
                                      _ptr(probs), pstride, _stream(stream))
    _check(st, "drs_row_stats_noalloc")


def drs_row_stats_seeds_workspace_bytes(rows: int, vocab: int, n_seeds: int) -> int:
    return int(load().drs_row_stats_seeds_workspace_bytes(rows, vocab, n_seeds))


def drs_row_stats_seeds(logits, temps, canvas_len, seeds, argmax, samples, entropy,
                        probs_dtype=DRS_PROBS_NONE, probs=None, workspace=None, stream=None,
                        row0=0):
    """Launch drs_row_stats_seeds: `seeds` a sequence of ints (host), samples
    an int64 CUDA tensor [len(seeds), rows]."""
    rows, vocab = logits.shape
    n = len(seeds)
    keys = (ctypes.c_uint64 * max(n, 1))(*[int(x) & (2**64 - 1) for x in seeds])
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    pstride = 0 if probs is None else probs.stride(0)
    st = load().drs_row_stats_seeds(_ptr(logits), rows, vocab, _row_stride(logits), _ptr(temps),
                                    canvas_len, ctypes.cast(keys, ctypes.c_void_p), n, row0,
                                    _ptr(argmax), _ptr(samples), _ptr(entropy), probs_dtype,
                                    _ptr(probs), pstride, _ptr(workspace), ws_bytes,
                                    _stream(stream))
    _check(st, "drs_row_stats_seeds")


def drs_row_stats_topk_workspace_bytes(rows: int, vocab: int, k: int) -> int:
    return int(load().drs_row_stats_topk_workspace_bytes(rows, vocab, k))


def drs_row_stats_topk(logits, temps, canvas_len, seed, argmax, sample, entropy, probs_dtype,
                       probs, keep, k, out_ids, out_logprobs, workspace=None, stream=None, row0=0):
    """Launch drs_row_stats_topk (row statistics and the top-k logprobs of
    converged rows, one read of the logits) on torch CUDA tensors."""
    rows, vocab = logits.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    pstride = 0 if probs is None else probs.stride(0)
    st = load().drs_row_stats_topk(_ptr(logits), rows, vocab, _row_stride(logits), _ptr(temps),
                                   canvas_len, seed & (2**64 - 1), row0, _ptr(argmax),
                                   _ptr(sample), _ptr(entropy), probs_dtype, _ptr(probs), pstride,
                                   _ptr(keep), k, _ptr(out_ids), _ptr(out_logprobs),
                                   _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "drs_row_stats_topk")


def drs_topk_workspace_bytes(rows: int, vocab: int, k: int) -> int:
    return int(load().drs_topk_workspace_bytes(rows, vocab, k))


def drs_topk_logprobs(logits, temps, canvas_len, keep, k, out_ids, out_logprobs,
                      workspace=None, stream=None):
    rows, vocab = logits.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().drs_topk_logprobs(_ptr(logits), rows, vocab, _row_stride(logits), _ptr(temps),
                                  canvas_len, _ptr(keep), k, _ptr(out_ids), _ptr(out_logprobs),
                                  _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "drs_topk_logprobs")


def drs_stash_workspace_bytes(requests: int, canvas_len: int, vocab: int, num_topk: int) -> int:
    return load().drs_stash_workspace_bytes(requests, canvas_len, vocab, num_topk)


def drs_stash_converged_logprobs(logits, canvas_len, src, slots, keep, valid, temps, num_topk,
                                 num_token_ids, token_ids, out_ids, out_logprobs, out_ranks,
                                 logits_mode, workspace=None, stream=None):
    """out_ids / out_logprobs: [out_slots, canvas_len, width]; out_ranks:
    [out_slots, canvas_len]; token_ids: None or int32 [requests, n]."""
    rows, vocab = logits.shape
    requests = src.shape[0]
    out_slots, _, width = out_ids.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    ids_stride = token_ids.stride(0) if token_ids is not None else 0
    st = load().drs_stash_converged_logprobs(
        _ptr(logits), rows, vocab, _row_stride(logits), canvas_len, requests, _ptr(src),
        _ptr(slots), _ptr(keep), _ptr(valid), _ptr(temps), num_topk, _ptr(num_token_ids),
        _ptr(token_ids), ids_stride, out_slots, width, _ptr(out_ids), _ptr(out_logprobs),
        _ptr(out_ranks), 1 if logits_mode else 0, _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "drs_stash_converged_logprobs")


def drs_philox_gumbel(seed, row0, rows, vocab, out_bits=None, out_gumbel=None, stream=None):
    st = load().drs_philox_gumbel(seed & (2**64 - 1), row0, rows, vocab, _ptr(out_bits),
                                  _ptr(out_gumbel), _stream(stream))
    _check(st, "drs_philox_gumbel")


def drs_scaled_logits(logits, temp: float, out, stream=None):
    """out = logits / max(temp, 1e-10) elementwise (contiguous fp32 tensors)."""
    assert logits.is_contiguous() and out.is_contiguous() and out.numel() == logits.numel()
    st = load().drs_scaled_logits(_ptr(logits), logits.numel(), temp, _ptr(out), _stream(stream))
    _check(st, "drs_scaled_logits")


# The token operators check what the library cannot: the types, devices and
# lengths of the arrays (ValueError). Sizes, strides and alignment are the
# library's own checks (DrsError).

_dtype_codes = {}


def _dtype_code(t, name: str) -> int:
    if not _dtype_codes:
        import torch
        _dtype_codes.update({torch.float32: DRS_DTYPE_FP32, torch.bfloat16: DRS_DTYPE_BF16,
                             torch.float16: DRS_DTYPE_FP16})
    code = _dtype_codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: fp32, bf16 or fp16 expected, got {t.dtype}")
    return code


def _raw_stream(stream, gpu: int) -> int:
    """The stream of a call on tensors of this GPU, which has to be the current
    device, where the library launches (torch.cuda.current_stream() alone takes
    3 us, more than a launch)."""
    import torch
    current = torch._C._cuda_getDevice()  # 0.1 us; torch.cuda.current_device() 0.2
    if gpu != current:
        raise ValueError(f"tensors on cuda:{gpu}, but the current device is cuda:{current}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(gpu)
    if stream.device_index != gpu:
        raise ValueError(f"stream: of cuda:{gpu} expected, got one of cuda:{stream.device_index}")
    return stream.cuda_stream


def _vector(t, name: str, dtype, n: int, gpu: int) -> int:
    """The address of a contiguous tensor of n elements of this type on this
    GPU."""
    if t.dtype is dtype and t.numel() == n and t.get_device() == gpu and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: contiguous {dtype} with {n} elements on cuda:{gpu} expected, got {t.dtype} "
                     f"{tuple(t.shape)} on {t.device}, strides {t.stride()}")


def _rows(t, name: str, gpu: int = -1) -> int:
    """The row stride of a 2-D tensor with unit column stride on a GPU (this
    one when given)."""
    if t.dim() != 2 or not t.is_cuda or (gpu >= 0 and t.get_device() != gpu):
        raise ValueError(f"{name}: 2-D on {f'cuda:{gpu}' if gpu >= 0 else 'a CUDA device'} expected, got {t.dim()}-D "
                         f"on {t.device}")
    rows, columns = t.shape
    step, unit = t.stride()
    if rows == 0 or columns == 0:
        return columns
    if unit != 1 and columns > 1:
        raise ValueError(f"{name}: unit column stride expected, got strides {t.stride()}")
    return step if rows > 1 else max(step, columns)


def drs_verify_drafts(target, draft, draft_tokens, cu_drafts, accept_u, sample_u, out_tokens,
                      out_accepted, stream=None):
    """Launch drs_verify_drafts: target [drafts + requests, vocab], draft
    [drafts, vocab] or None, out_tokens int64 [requests, max_drafts + 1]."""
    import torch
    target_stride = _rows(target, "target")
    gpu = target.get_device()
    target_rows, vocab = target.shape
    drafts, requests = draft_tokens.numel(), sample_u.numel()
    draft_ptr, draft_code, draft_stride = None, 0, 0
    if draft is not None:
        draft_stride = _rows(draft, "draft", gpu)
        draft_code = _dtype_code(draft, "draft")
        if draft.shape != (drafts, vocab):
            raise ValueError(f"draft: {(drafts, vocab)} expected, got {tuple(draft.shape)}")
        draft_ptr = draft.data_ptr()
    if out_tokens.dim() != 2 or out_tokens.shape[0] != requests or out_tokens.shape[1] < 1:
        raise ValueError(f"out_tokens: [{requests}, max_drafts + 1] expected, got {tuple(out_tokens.shape)}")
    width = out_tokens.shape[1]
    st = load().drs_verify_drafts(
        target.data_ptr(), _dtype_code(target, "target"), target_rows, target_stride, draft_ptr, draft_code, drafts,
        draft_stride, vocab, _vector(draft_tokens, "draft_tokens", torch.int64, drafts, gpu),
        _vector(cu_drafts, "cu_drafts", torch.int32, requests + 1, gpu), requests, width - 1,
        _vector(accept_u, "accept_u", torch.float32, drafts, gpu),
        _vector(sample_u, "sample_u", torch.float32, requests, gpu),
        _vector(out_tokens, "out_tokens", torch.int64, requests * width, gpu),
        _vector(out_accepted, "out_accepted", torch.int32, requests, gpu), _raw_stream(stream, gpu))
    _check(st, "drs_verify_drafts")


def drs_map_slots(lens, new_lens, held, block_table, block_size: int, free_ring, ring_state, out_cu,
                  out_request, out_position, out_slot, out_held, out_ring_state, out_lacking,
                  stream=None):
    """Launch drs_map_slots: int32 lengths [requests], block_table int32
    [requests, max_blocks] (any row stride); the token arrays' length is the
    capacity. block_table and free_ring are updated in place; out_held and
    out_ring_state may be held and ring_state."""
    import torch
    i32, i64 = torch.int32, torch.int64
    requests, capacity, ring = lens.numel(), out_request.numel(), free_ring.numel()
    table_stride = _rows(block_table, "block_table")
    gpu = block_table.get_device()
    if block_table.dtype is not i32 or block_table.shape[0] != requests:
        raise ValueError(f"block_table: int32 [{requests}, max_blocks] expected, got {block_table.dtype} "
                         f"{tuple(block_table.shape)}")
    st = load().drs_map_slots(
        _vector(lens, "lens", i32, requests, gpu), _vector(new_lens, "new_lens", i32, requests, gpu),
        _vector(held, "held", i32, requests, gpu), requests, block_size, block_table.data_ptr(), table_stride,
        block_table.shape[1], _vector(free_ring, "free_ring", i32, ring, gpu), ring,
        _vector(ring_state, "ring_state", i64, 2, gpu), capacity, _vector(out_cu, "out_cu", i32, requests + 1, gpu),
        _vector(out_request, "out_request", i32, capacity, gpu),
        _vector(out_position, "out_position", i32, capacity, gpu), _vector(out_slot, "out_slot", i64, capacity, gpu),
        _vector(out_held, "out_held", i32, requests, gpu),
        _vector(out_ring_state, "out_ring_state", i64, 2, gpu),
        _vector(out_lacking, "out_lacking", i32, 1, gpu), _raw_stream(stream, gpu))
    _check(st, "drs_map_slots")


def _id_bits(ids) -> int:
    import torch
    if ids.dtype is torch.int64:
        return 64
    if ids.dtype is torch.int32:
        return 32
    raise ValueError(f"ids: int32 or int64 expected, got {ids.dtype}")


def _no_history(a, b, what: str, gradient: str = "the table's gradient is embed_tokens_grad"):
    """The calls leave no autograd history: refused rather than cut off
    silently (torch's own functions with `out` do the same)."""
    import torch
    if (a.requires_grad or b.requires_grad) and torch.is_grad_enabled():
        raise ValueError(f"{what}: a tensor requires a gradient, and the call leaves no history; detach it or call "
                         f"under torch.no_grad() ({gradient})")


def drs_embed_tokens(table, ids, scale: float, out, stream=None):
    """Launch drs_embed_tokens: table [vocab, width], ids int32 or int64
    [tokens], out [tokens, width] of the table's type."""
    _no_history(table, out, "drs_embed_tokens")
    gpu = table.get_device()
    table_stride, out_stride = _rows(table, "table"), _rows(out, "out", gpu)
    vocab, width = table.shape
    tokens = ids.numel()
    if out.dtype is not table.dtype or out.shape != (tokens, width):
        raise ValueError(f"out: {table.dtype} {(tokens, width)} expected, got {out.dtype} {tuple(out.shape)}")
    st = load().drs_embed_tokens(table.data_ptr(), _dtype_code(table, "table"), vocab, width, table_stride,
                                 _vector(ids, "ids", ids.dtype, tokens, gpu), _id_bits(ids), tokens, scale,
                                 out.data_ptr(), out_stride, _raw_stream(stream, gpu))
    _check(st, "drs_embed_tokens")


@functools.lru_cache(maxsize=256)
def drs_embed_tokens_grad_workspace_bytes(tokens: int, vocab: int, width: int) -> int:
    return int(load().drs_embed_tokens_grad_workspace_bytes(tokens, vocab, width))


def drs_embed_tokens_grad(grad_out, ids, scale: float, accumulate: bool, grad_table, workspace=None,
                          stream=None):
    """Launch drs_embed_tokens_grad: grad_out [tokens, width], grad_table
    [vocab, width] (each fp32, bf16 or fp16)."""
    _no_history(grad_out, grad_table, "drs_embed_tokens_grad")
    gpu = grad_out.get_device()
    grad_stride, table_stride = _rows(grad_out, "grad_out"), _rows(grad_table, "grad_table", gpu)
    vocab, width = grad_table.shape
    tokens = ids.numel()
    if grad_out.shape != (tokens, width):
        raise ValueError(f"grad_out: {(tokens, width)} expected, got {tuple(grad_out.shape)}")
    ws, ws_bytes = None, 0
    if workspace is not None:
        if workspace.get_device() != gpu or not workspace.is_contiguous():
            raise ValueError(f"workspace: contiguous on cuda:{gpu} expected, got {workspace.device}")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = load().drs_embed_tokens_grad(grad_out.data_ptr(), _dtype_code(grad_out, "grad_out"), tokens, width,
                                      grad_stride, _vector(ids, "ids", ids.dtype, tokens, gpu), _id_bits(ids), scale,
                                      1 if accumulate else 0, grad_table.data_ptr(),
                                      _dtype_code(grad_table, "grad_table"), vocab, table_stride, ws, ws_bytes,
                                      _raw_stream(stream, gpu))
    _check(st, "drs_embed_tokens_grad")


# The scoring operators and dropout check the same in fewer calls: their smallest
# kernels take 2 us, and every question to a tensor 0.07 to 0.1.

def _matrix(t, name: str, shape, gpu: int):
    """(address, type's code, row stride) of a tensor of this 2-D shape with
    unit column stride on this GPU."""
    code = _dtype_codes.get(t.dtype)
    if code is None:
        code = _dtype_code(t, name)
    if t.shape != shape or t.get_device() != gpu or gpu < 0:
        raise ValueError(f"{name}: {tuple(shape)} on {f'cuda:{gpu}' if gpu >= 0 else 'a CUDA device'} expected, got "
                         f"{tuple(t.shape)} on {t.device}")
    rows, columns = shape
    step, unit = t.stride()
    if unit != 1 and columns > 1 and rows > 0:
        raise ValueError(f"{name}: unit column stride expected, got strides {t.stride()}")
    return t.data_ptr(), code, step if rows > 1 and columns > 0 else max(step, columns)


def _shape2(t, name: str):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: 2-D expected, got {tuple(shape)}")
    return shape


def _ids_and_temps(ids, temps, rows: int, canvas_len: int, gpu: int):
    import torch
    bits = 64 if ids.dtype is torch.int64 else _id_bits(ids)
    if canvas_len < 1:
        raise ValueError(f"canvas_len: at least 1 expected, got {canvas_len}")
    return (_vector(ids, "ids", ids.dtype, rows, gpu), bits,
            None if temps is None else _vector(temps, "temps", torch.float32, -(-rows // canvas_len), gpu))


def drs_token_logprobs(logits, ids, temps, canvas_len: int, out_logprob, out_entropy, out_rank, out_norm, out_ids,
                       out_logprobs, stream=None):
    """Launch drs_token_logprobs: logits [rows, vocab], ids int32 or int64
    [rows]; k is the width of out_ids [rows, k]. out_entropy, out_rank and
    out_norm may be None, out_ids and out_logprobs too (k = 0)."""
    import torch
    f32, i32 = torch.float32, torch.int32
    if logits.requires_grad or out_logprob.requires_grad:
        _no_history(logits, out_logprob, "drs_token_logprobs", "the logits' gradient is token_logprobs_grad")
    shape, gpu = _shape2(logits, "logits"), logits.get_device()
    rows, vocab = shape
    ptr, code, stride = _matrix(logits, "logits", shape, gpu)
    k, top_ids, top_logprobs = 0, None, None
    if out_ids is not None and out_logprobs is not None:
        if out_ids.dim() != 2:
            raise ValueError(f"out_ids: [{rows}, k] expected, got {tuple(out_ids.shape)}")
        k = out_ids.shape[1]
        top_ids = _vector(out_ids, "out_ids", i32, rows * k, gpu)
        top_logprobs = _vector(out_logprobs, "out_logprobs", f32, rows * k, gpu)
    elif out_ids is not None or out_logprobs is not None:
        raise ValueError("out_ids and out_logprobs: both or neither expected")
    ids_ptr, bits, temps_ptr = _ids_and_temps(ids, temps, rows, canvas_len, gpu)
    st = load().drs_token_logprobs(
        ptr, code, rows, vocab, stride, ids_ptr, bits, temps_ptr, canvas_len, k,
        _vector(out_logprob, "out_logprob", f32, rows, gpu),
        None if out_entropy is None else _vector(out_entropy, "out_entropy", f32, rows, gpu),
        None if out_rank is None else _vector(out_rank, "out_rank", i32, rows, gpu),
        None if out_norm is None else _vector(out_norm, "out_norm", f32, 2 * rows, gpu), top_ids, top_logprobs,
        _raw_stream(stream, gpu))
    if st != DRS_OK:
        _check(st, "drs_token_logprobs")


def drs_token_logprobs_grad(logits, ids, temps, canvas_len: int, norm, entropy, grad_logprob, grad_entropy, grad,
                            stream=None):
    """Launch drs_token_logprobs_grad: grad [rows, vocab] (fp32, bf16 or fp16,
    or logits itself); grad_logprob or grad_entropy may be None, entropy
    without grad_entropy too."""
    import torch
    f32 = torch.float32
    if logits.requires_grad or grad.requires_grad:
        _no_history(logits, grad, "drs_token_logprobs_grad", "there is no second derivative")
    shape, gpu = _shape2(logits, "logits"), logits.get_device()
    rows, vocab = shape
    ptr, code, stride = _matrix(logits, "logits", shape, gpu)
    grad_ptr, grad_code, grad_stride = _matrix(grad, "grad", shape, gpu)
    ids_ptr, bits, temps_ptr = _ids_and_temps(ids, temps, rows, canvas_len, gpu)
    st = load().drs_token_logprobs_grad(
        ptr, code, rows, vocab, stride, ids_ptr, bits, temps_ptr, canvas_len, _vector(norm, "norm", f32, 2 * rows, gpu),
        None if entropy is None else _vector(entropy, "entropy", f32, rows, gpu),
        None if grad_logprob is None else _vector(grad_logprob, "grad_logprob", f32, rows, gpu),
        None if grad_entropy is None else _vector(grad_entropy, "grad_entropy", f32, rows, gpu),
        grad_ptr, grad_code, grad_stride, _raw_stream(stream, gpu))
    if st != DRS_OK:
        _check(st, "drs_token_logprobs_grad")


def _seed(seed, gpu: int):
    """(host seed, address of the device's): a whole number, or an int64 or
    uint64 tensor of one element on the GPU."""
    if isinstance(seed, int):
        return seed & (2**64 - 1), None
    import torch
    dtype = getattr(seed, "dtype", None)
    if dtype is not torch.int64 and dtype is not torch.uint64:
        raise ValueError(f"seed: an int or one int64 on the GPU expected, got {type(seed).__name__} {dtype}")
    return 0, _vector(seed, "seed", dtype, 1, gpu)


def drs_dropout(x, residual, p: float, seed, row0: int, out, stream=None):
    """Launch drs_dropout: x and out [rows, width], residual None or of out's
    type and shape; seed an int or an int64 tensor of one element on the GPU."""
    if x.requires_grad or out.requires_grad:
        _no_history(x, out, "drs_dropout", "the gradient is dropout_grad")
    shape, gpu = _shape2(x, "x"), x.get_device()
    x_ptr, x_code, x_stride = _matrix(x, "x", shape, gpu)
    out_ptr, out_code, out_stride = _matrix(out, "out", shape, gpu)
    residual_ptr, residual_stride = None, 0
    if residual is not None:
        if residual.requires_grad:
            _no_history(residual, out, "drs_dropout", "the residual's gradient is the output's")
        residual_ptr, residual_code, residual_stride = _matrix(residual, "residual", shape, gpu)
        if residual_code != out_code:
            raise ValueError(f"residual: {out.dtype} expected, got {residual.dtype}")
    key, device_key = _seed(seed, gpu)
    st = load().drs_dropout(x_ptr, x_code, shape[0], shape[1], x_stride, residual_ptr, residual_stride, p, key, device_key,
                            row0, out_ptr, out_code, out_stride, _raw_stream(stream, gpu))
    if st != DRS_OK:
        _check(st, "drs_dropout")


def drs_dropout_grad(grad_out, p: float, seed, row0: int, grad_x, stream=None):
    """Launch drs_dropout_grad: grad_out and grad_x [rows, width] (each fp32,
    bf16 or fp16); seed as drs_dropout."""
    if grad_out.requires_grad or grad_x.requires_grad:
        _no_history(grad_out, grad_x, "drs_dropout_grad", "the gradient of a gradient is dropout_grad again")
    shape, gpu = _shape2(grad_out, "grad_out"), grad_out.get_device()
    grad_ptr, grad_code, grad_stride = _matrix(grad_out, "grad_out", shape, gpu)
    x_ptr, x_code, x_stride = _matrix(grad_x, "grad_x", shape, gpu)
    key, device_key = _seed(seed, gpu)
    st = load().drs_dropout_grad(grad_ptr, grad_code, shape[0], shape[1], grad_stride, p, key, device_key, row0, x_ptr,
                                 x_code, x_stride, _raw_stream(stream, gpu))
    if st != DRS_OK:
        _check(st, "drs_dropout_grad")


KERNEL_NAMES = ("split_prep", "split_pass1", "split_merge", "split_pass2", "split_cluster",
                "split_finish")


def drs_kernel_timing(enable: bool) -> None:
    """Measurement hook: record CUDA events around the row kernels of every
    following call on the current device (see include/drs.h)."""
    _check(load().drs_kernel_timing(1 if enable else 0), "drs_kernel_timing")


def drs_kernel_times():
    """Average ms of each row kernel over the calls recorded since timing was
    switched on: ({kernel name: ms}, number of calls averaged)."""
    out = (ctypes.c_float * len(KERNEL_NAMES))()
    calls = ctypes.c_int32(0)
    _check(load().drs_kernel_times(ctypes.cast(out, ctypes.c_void_p), len(KERNEL_NAMES),
                                   ctypes.cast(ctypes.pointer(calls), ctypes.c_void_p)),
           "drs_kernel_times")
    return dict(zip(KERNEL_NAMES, (float(v) for v in out))), int(calls.value)


def drs_test_inject_fault(code: int) -> None:
    """Test hook: in the next row-statistics call a CTA never fills its first
    stage, so that the bounded waits on it run out (see include/drs.h)."""
    load().drs_test_inject_fault(code)


def drs_test_two_pass(on: bool) -> None:
    """Test hook: every following row-statistics call takes the two passes
    over the logits instead of the one-read cluster kernel (see
    include/drs.h)."""
    load().drs_test_two_pass(1 if on else 0)


def cluster_rows(rows: int, vocab: int, k: int, n_seeds: int = 1, probs_dtype: int = DRS_PROBS_BF16,
                 stats: bool = True):
    """How a row-statistics call of these sizes shares its rows on the
    current device (drs_row_split_plan): None when it takes the two passes
    alone, else a dict with the rows of the cluster kernel ("head"), of the
    two passes beside it ("tail"), the cluster size, the clusters resident
    at once and the SMs they leave free."""
    head, size, ncl, free = ctypes.c_int64(0), ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_int32(0)
    _check(load().drs_row_split_plan(rows, vocab, k, n_seeds, probs_dtype, 1 if stats else 0,
                                     ctypes.byref(head), ctypes.byref(size), ctypes.byref(ncl),
                                     ctypes.byref(free)), "drs_row_split_plan")
    if size.value == 0:
        return None
    return {"head": int(head.value), "tail": int(rows - head.value), "cluster_size": int(size.value),
            "clusters": int(ncl.value), "free_sms": int(free.value)}


def drs_get_device_error(stream=None) -> int:
    return int(load().drs_get_device_error(_stream(stream)))


# ------------------------------------------------------------- conveniences

_workspaces = {}


def workspace(nbytes: int, device):
    """A cached device workspace of at least nbytes (256-byte aligned)."""
    import torch
    key = (str(device), nbytes)
    ws = _workspaces.get(key)
    if ws is None:
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def row_stats(logits, temps, canvas_len: int, seed: int, probs_dtype=None, stream=None,
              row0: int = 0):
    """Allocate outputs and run drs_row_stats; returns (argmax, sample,
    entropy, probs) like the page's sample_row_stats."""
    import torch
    rows, vocab = logits.shape
    dev = logits.device
    argmax = torch.empty(rows, dtype=torch.int64, device=dev)
    sample = torch.empty(rows, dtype=torch.int64, device=dev)
    entropy = torch.empty(rows, dtype=torch.float32, device=dev)
    code = {None: DRS_PROBS_NONE, torch.bfloat16: DRS_PROBS_BF16,
            torch.float16: DRS_PROBS_FP16}[probs_dtype]
    probs = None if probs_dtype is None else torch.empty(rows, vocab, dtype=probs_dtype, device=dev)
    if rows == 0:
        return argmax, sample, entropy, probs
    ws = workspace(drs_row_stats_workspace_bytes(rows, vocab), dev)
    drs_row_stats(logits, temps, canvas_len, seed, argmax, sample, entropy, code, probs, ws,
                  stream, row0)
    return argmax, sample, entropy, probs


def row_stats_seeds(logits, temps, canvas_len: int, seeds, probs_dtype=None, stream=None,
                    row0: int = 0):
    """Allocate outputs and run drs_row_stats_seeds; returns (argmax,
    samples [len(seeds), rows], entropy, probs)."""
    import torch
    rows, vocab = logits.shape
    dev = logits.device
    argmax = torch.empty(rows, dtype=torch.int64, device=dev)
    samples = torch.empty(len(seeds), rows, dtype=torch.int64, device=dev)
    entropy = torch.empty(rows, dtype=torch.float32, device=dev)
    code = {None: DRS_PROBS_NONE, torch.bfloat16: DRS_PROBS_BF16,
            torch.float16: DRS_PROBS_FP16}[probs_dtype]
    probs = None if probs_dtype is None else torch.empty(rows, vocab, dtype=probs_dtype, device=dev)
    if rows == 0:
        return argmax, samples, entropy, probs
    ws = workspace(drs_row_stats_seeds_workspace_bytes(rows, vocab, len(seeds)), dev)
    drs_row_stats_seeds(logits, temps, canvas_len, seeds, argmax, samples, entropy, code, probs,
                        ws, stream, row0)
    return argmax, samples, entropy, probs


def row_stats_topk(logits, temps, canvas_len: int, seed: int, keep, k: int, probs_dtype=None,
                   out_ids=None, out_logprobs=None, stream=None, row0: int = 0):
    """Allocate outputs and run drs_row_stats_topk; returns (argmax, sample,
    entropy, probs, out_ids, out_logprobs). Rows of unconverged slots keep
    the given (or -1 / NaN filled) top-k outputs."""
    import torch
    rows, vocab = logits.shape
    dev = logits.device
    argmax = torch.empty(rows, dtype=torch.int64, device=dev)
    sample = torch.empty(rows, dtype=torch.int64, device=dev)
    entropy = torch.empty(rows, dtype=torch.float32, device=dev)
    code = {None: DRS_PROBS_NONE, torch.bfloat16: DRS_PROBS_BF16,
            torch.float16: DRS_PROBS_FP16}[probs_dtype]
    probs = None if probs_dtype is None else torch.empty(rows, vocab, dtype=probs_dtype, device=dev)
    if out_ids is None:
        out_ids = torch.full((rows, k), -1, dtype=torch.int32, device=dev)
    if out_logprobs is None:
        out_logprobs = torch.full((rows, k), float("nan"), dtype=torch.float32, device=dev)
    if rows == 0:
        return argmax, sample, entropy, probs, out_ids, out_logprobs
    ws = workspace(max(drs_row_stats_topk_workspace_bytes(rows, vocab, k),
                       drs_row_stats_workspace_bytes(rows, vocab)), dev)
    drs_row_stats_topk(logits, temps, canvas_len, seed, argmax, sample, entropy, code, probs,
                       keep, k, out_ids, out_logprobs, ws, stream, row0)
    return argmax, sample, entropy, probs, out_ids, out_logprobs


def topk_logprobs(logits, temps, canvas_len: int, keep, k: int, out_ids=None,
                  out_logprobs=None, stream=None):
    """Top-k ids and logprobs of the rows of kept slots (other rows of the
    given outputs are left as they are)."""
    import torch
    rows, vocab = logits.shape
    dev = logits.device
    if out_ids is None:
        out_ids = torch.full((rows, k), -1, dtype=torch.int32, device=dev)
    if out_logprobs is None:
        out_logprobs = torch.full((rows, k), float("nan"), dtype=torch.float32, device=dev)
    ws = workspace(drs_topk_workspace_bytes(rows, vocab, k), dev)
    drs_topk_logprobs(logits, temps, canvas_len, keep, k, out_ids, out_logprobs, ws, stream)
    return out_ids, out_logprobs


def philox_gumbel(seed: int, row0: int, rows: int, vocab: int, device="cuda", stream=None):
    import torch
    bits = torch.empty(rows, vocab, dtype=torch.int32, device=device)
    g = torch.empty(rows, vocab, dtype=torch.float32, device=device)
    drs_philox_gumbel(seed, row0, rows, vocab, bits, g, stream)
    return bits, g


def stash_converged_logprobs(logits, canvas_len: int, src, slots, keep, valid, temps,
                             num_topk: int, num_token_ids=None, token_ids=None, out_ids=None,
                             out_logprobs=None, out_ranks=None, out_slots: int | None = None,
                             width: int | None = None, logits_mode: bool = False, stream=None):
    """The stash (see drs_stash_converged_logprobs); outputs allocated when
    not given, filled with -1 / NaN / -1 where the stash does not write."""
    import torch
    dev = logits.device
    if out_ids is None:
        out_slots = int(src.shape[0]) if out_slots is None else out_slots
        width = num_topk + 1 if width is None else width
        out_ids = torch.full((out_slots, canvas_len, width), -1, dtype=torch.int32, device=dev)
    if out_logprobs is None:
        out_logprobs = torch.full(out_ids.shape, float("nan"), dtype=torch.float32, device=dev)
    if out_ranks is None:
        out_ranks = torch.full(out_ids.shape[:2], -1, dtype=torch.int32, device=dev)
    ws = workspace(drs_stash_workspace_bytes(int(src.shape[0]), canvas_len, logits.shape[1],
                                             num_topk), dev)
    drs_stash_converged_logprobs(logits, canvas_len, src, slots, keep, valid, temps, num_topk,
                                 num_token_ids, token_ids, out_ids, out_logprobs, out_ranks,
                                 logits_mode, ws, stream)
    return out_ids, out_logprobs, out_ranks


def _allocate_on(stream):
    """Where a call on `stream` allocates: the caching allocator hands memory
    on in the order of the stream that it was allocated on."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    return torch.cuda.stream(stream)


class _StreamWorkspace:
    """The workspace of one stream's calls, and the lock under which a call
    has it."""

    __slots__ = ("lock", "buffer")

    def __init__(self):
        self.lock, self.buffer = threading.RLock(), None

    def at_least(self, nbytes: int, gpu: int):
        """Replaced by a larger one when needed: both belong to the stream, so
        what still runs on it is done with the old one before its memory is
        used again."""
        if self.buffer is None or self.buffer.numel() < nbytes:
            self.buffer = _new_workspace(nbytes, gpu)
        return self.buffer


# What is kept at most: workspaces of up to 4 MB of 16 streams. A larger one's
# allocation hides behind its call's time on the GPU (accumulating calls with 4.1 to
# 4.4 MB: 1024 x 4200 16.5 us kept, 16.6 not; 4096 x 1088 19.4, 19.6; 64 x 70000
# alone 12.4, 16.5). The allocator takes back what is dropped in its stream's order.
_KEPT_BYTES = 4 << 20
_KEPT_STREAMS = 16
_stream_workspaces = {}


def _new_workspace(nbytes: int, gpu: int):
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{gpu}")


def verify_drafts(target_probs, draft_tokens, cu_drafts, accept_u, sample_u, max_drafts: int,
                  draft_probs=None, out_tokens=None, out_accepted=None, stream=None):
    """Verify drafted tokens against the target's probabilities (see
    drs_verify_drafts); returns (tokens int64 [requests, max_drafts + 1]: the
    accepted drafts, one more token, then -1; accepted int32 [requests])."""
    import torch
    requests = sample_u.numel()
    if max_drafts < 0 or (out_tokens is not None and out_tokens.shape != (requests, max_drafts + 1)):
        raise ValueError(f"out_tokens: [{requests}, max_drafts + 1] with max_drafts {max_drafts} expected")
    if out_tokens is None or out_accepted is None:
        with _allocate_on(stream):
            if out_tokens is None:
                out_tokens = torch.empty(requests, max_drafts + 1, dtype=torch.int64, device=target_probs.device)
            if out_accepted is None:
                out_accepted = torch.empty(requests, dtype=torch.int32, device=target_probs.device)
    drs_verify_drafts(target_probs, draft_probs, draft_tokens, cu_drafts, accept_u, sample_u, out_tokens,
                      out_accepted, stream)
    return out_tokens, out_accepted


def map_slots(lens, new_lens, held, block_table, block_size: int, free_ring, ring_state, capacity: int,
              out=None, stream=None):
    """Block tables and slot maps from the requests' lengths (see
    drs_map_slots). Returns `out`: (cu, request, position, slot, held,
    ring_state, lacking), allocated when not given; block_table and
    free_ring are updated in place."""
    import torch
    if out is None:
        dev, requests = lens.device, lens.numel()
        i32, i64 = dict(dtype=torch.int32, device=dev), dict(dtype=torch.int64, device=dev)
        with _allocate_on(stream):
            out = (torch.empty(requests + 1, **i32), torch.empty(capacity, **i32), torch.empty(capacity, **i32),
                   torch.empty(capacity, **i64), torch.empty(requests, **i32), torch.empty(2, **i64),
                   torch.empty(1, **i32))
    elif out[1].numel() != capacity:
        raise ValueError(f"out: token arrays of {capacity} entries expected, got {out[1].numel()}")
    drs_map_slots(lens, new_lens, held, block_table, block_size, free_ring, ring_state, *out, stream=stream)
    return out


def embed_tokens(table, ids, scale: float = 1.0, out=None, stream=None):
    """scale * table[ids] (see drs_embed_tokens); rows of ids outside the
    vocabulary are 0. No autograd history: a table that requires a gradient
    is refused while autograd records, and its gradient is embed_tokens_grad."""
    import torch
    if out is None:
        with _allocate_on(stream):
            out = torch.empty(ids.numel(), table.shape[1], dtype=table.dtype, device=table.device)
    drs_embed_tokens(table, ids, scale, out, stream)
    return out


def embed_tokens_grad(grad_out, ids, scale: float, grad_table, accumulate: bool = False, stream=None):
    """The gradient of embed_tokens with respect to its table, written (or
    added) into grad_table [vocab, width], which is returned (see
    drs_embed_tokens_grad)."""
    if grad_table.dim() != 2:
        raise ValueError(f"grad_table: [vocab, width] expected, got {tuple(grad_table.shape)}")
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return embed_tokens_grad(grad_out, ids, scale, grad_table, accumulate)
    size, gpu = drs_embed_tokens_grad_workspace_bytes(ids.numel(), *grad_table.shape), grad_out.get_device()
    if gpu < 0 or size == 0:
        drs_embed_tokens_grad(grad_out, ids, scale, accumulate, grad_table)
    elif size > _KEPT_BYTES or torch.cuda.is_current_stream_capturing():  # captured: one of the graph's own
        drs_embed_tokens_grad(grad_out, ids, scale, accumulate, grad_table, _new_workspace(size, gpu))
    else:
        # Kept per stream: a call of 16 tokens takes 10.7 us so, and 16.2 with a
        # workspace from the allocator. Threads that share the stream take
        # turns, each until its launches are all on the stream.
        key = (gpu, _raw_stream(None, gpu))
        kept = _stream_workspaces.get(key)
        if kept is None:
            if len(_stream_workspaces) >= _KEPT_STREAMS:
                _stream_workspaces.clear()
            kept = _stream_workspaces.setdefault(key, _StreamWorkspace())
        with kept.lock:
            drs_embed_tokens_grad(grad_out, ids, scale, accumulate, grad_table, kept.at_least(size, gpu))
    return grad_table


def token_logprobs(logits, ids, k: int = 0, temps=None, canvas_len: int = 1, out=None, stream=None):
    """Log probabilities of the rows' tokens under softmax(logits / T), with
    entropy, rank and the k largest alternatives (see drs_token_logprobs).
    Returns `out`: (logprob, entropy, rank, norm [rows, 2], top_ids [rows, k],
    top_logprobs [rows, k]), allocated when not given. No autograd history:
    the logits' gradient is token_logprobs_grad, which takes norm and entropy;
    there is none for temps."""
    if out is None:
        import torch
        dev, rows = logits.device, logits.shape[0]
        f32, i32 = dict(dtype=torch.float32, device=dev), dict(dtype=torch.int32, device=dev)
        with _allocate_on(stream):
            out = (torch.empty(rows, **f32), torch.empty(rows, **f32), torch.empty(rows, **i32),
                   torch.empty(rows, 2, **f32), torch.empty(rows, k, **i32), torch.empty(rows, k, **f32))
    elif out[4] is None:
        if k != 0:
            raise ValueError(f"out: [rows, {k}] alternatives expected, got none")
    elif out[4].shape != (logits.shape[0], k):
        raise ValueError(f"out: [{logits.shape[0]}, {k}] alternatives expected, got {tuple(out[4].shape)}")
    drs_token_logprobs(logits, ids, temps, canvas_len, *out, stream=stream)
    return out


def token_logprobs_grad(logits, ids, norm, grad_logprob, entropy=None, grad_entropy=None, temps=None,
                        canvas_len: int = 1, out=None, stream=None):
    """The gradient of token_logprobs' logprob and entropy with respect to the
    logits, from its norm (and entropy, with grad_entropy), written into out
    [rows, vocab] (allocated in the logits' type when not given; logits
    itself is allowed), which is returned (see drs_token_logprobs_grad)."""
    if out is None:
        import torch
        with _allocate_on(stream):
            out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    drs_token_logprobs_grad(logits, ids, temps, canvas_len, norm, entropy, grad_logprob, grad_entropy, out, stream)
    return out


def dropout(x, p: float, seed, residual=None, row0: int = 0, out=None, stream=None):
    """Dropout of x [rows, width], added to the residual when one is given
    (see drs_dropout): the mask follows from seed (an int, or an int64 tensor
    of one element on the GPU), row0 and the place, and is not stored. out:
    of the residual's type, or x's, when not given. No autograd history: the
    gradient is dropout_grad."""
    if out is None:
        import torch
        with _allocate_on(stream):
            out = torch.empty(x.shape, dtype=x.dtype if residual is None else residual.dtype, device=x.device)
    drs_dropout(x, residual, p, seed, row0, out, stream)
    return out


def dropout_grad(grad_out, p: float, seed, row0: int = 0, out=None, stream=None):
    """The gradient of dropout with respect to x, from the p, seed and row0 of
    the forward call, written into out (allocated in grad_out's type when not
    given; grad_out itself is allowed), which is returned."""
    if out is None:
        import torch
        with _allocate_on(stream):
            out = torch.empty(grad_out.shape, dtype=grad_out.dtype, device=grad_out.device)
    drs_dropout_grad(grad_out, p, seed, row0, out, stream)
    return out
