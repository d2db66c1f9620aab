"""ctypes binding of the spec_verify C ABI (include/spec_verify.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, their device pointers and the current CUDA stream are passed to
the library, and a non-OK status raises.  Every step of verification runs in
the library's kernels; there is no fallback.  torch is used for allocation
(outputs, workspace) and for the stream handle.  The operators around the
verification do the same from C++ (csrc/torch_ops.cpp).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading
from dataclasses import dataclass

import torch

from . import build as _build

SPEC_OK, SPEC_ERR_INVALID_ARG, SPEC_ERR_UNSUPPORTED, SPEC_ERR_CUDA, SPEC_ERR_WORKSPACE = range(5)
SPEC_F32, SPEC_BF16, SPEC_F16, SPEC_E4M3 = 0, 1, 2, 3
BADBIT = {"num_draft": 1, "temperature": 2, "draft_id": 4, "empty_row": 8, "no_probs": 16,
          "timeout": 32, "tree": 64, "page": 128}
MODE_BAD, MODE_GREEDY, MODE_RESIDUAL, MODE_BONUS, MODE_FALLBACK, MODE_TYPICAL = -1, 0, 1, 2, 3, 4
MAX_K = 31
# kernels of one call, in launch order: the request-by-request verifier
# (spec_verify_by_request, and spec_verify where verify_path() is 1), and the
# all-rows verifier (spec_verify_all_rows, and spec_verify where it is 0)
KERNELS = ("k_prep", "k_verify")
KERNELS_ALL_ROWS = ("k_plan", "k_row_stats", "k_accept_all", "k_sample", "k_emit")
N_KERNELS = len(KERNELS)
N_MARKS = 6  # events a profiled call records

_LOCK = threading.Lock()
_LIB = None
_OPS = None


class SpecVerifyError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)}")


def _declare(lib):
    vp, i32, u32, u64, i64, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint64,
                                  ctypes.c_int64, ctypes.c_size_t)
    lib.spec_status_str.restype = ctypes.c_char_p
    lib.spec_status_str.argtypes = [i32]
    lib.spec_verify_workspace_size.restype = sz
    lib.spec_verify_workspace_size.argtypes = [i32, i32, i32]
    lib.spec_verify_status_ptr.restype = vp
    lib.spec_verify_status_ptr.argtypes = [vp]
    common = [vp, i32, vp, vp, vp, vp, u64, i32, i32, i32, vp, vp, vp, sz, vp]
    lib.spec_verify.restype = i32
    lib.spec_verify.argtypes = common
    lib.spec_verify_ex.restype = i32
    lib.spec_verify_ex.argtypes = common + [u32, vp, vp, vp]
    lib.spec_verify_dev_seed.restype = i32
    lib.spec_verify_dev_seed.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp,
                                         sz, vp, u32, vp, vp, vp]
    lib.spec_verify_early_exit.restype = i32
    lib.spec_verify_early_exit.argtypes = common + [u32, vp, vp, vp, vp]
    lib.spec_verify_all_rows.restype = i32
    lib.spec_verify_all_rows.argtypes = common + [u32, vp, vp, vp, vp, vp]
    lib.spec_verify_by_request.restype = i32
    lib.spec_verify_by_request.argtypes = common + [u32, vp, vp, vp, vp, vp]
    lib.spec_verify_path.restype = i32
    lib.spec_verify_path.argtypes = [i32, i32, i32, i32]
    lib.spec_verify_lmhead_workspace_size.restype = sz
    lib.spec_verify_lmhead_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.spec_verify_lmhead.restype = i32
    lib.spec_verify_lmhead.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, u64, i32, i32, i32, vp, vp,
                                       vp, sz, vp, u32, vp, vp, vp]
    lib.spec_lmhead_logits.restype = i32
    lib.spec_lmhead_logits.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp]
    lib.spec_verify_tree_workspace_size.restype = sz
    lib.spec_verify_tree_workspace_size.argtypes = [i32, i32, i32]
    lib.spec_verify_tree.restype = i32
    lib.spec_verify_tree.argtypes = [vp, i32, vp, vp, vp, vp, vp, u64, i32, i32, i32, vp, vp, vp,
                                     vp, sz, vp, u32, vp, vp, vp]
    lib.spec_verify_typical.restype = i32
    lib.spec_verify_typical.argtypes = [vp, i32, vp, vp, vp, ctypes.c_float, u64, i32, i32, i32,
                                        vp, vp, vp, sz, vp, u32, vp, vp, vp]
    lib.spec_verify_profiled.restype = i32
    lib.spec_verify_profiled.argtypes = common + [vp]
    lib.spec_verify_host_small_bytes.restype = sz
    lib.spec_verify_host_small_bytes.argtypes = [i32, i32]
    lib.spec_verify_host.restype = i32
    lib.spec_verify_host.argtypes = [vp, i32, vp, vp, vp, vp, u64, i32, i32, i32, vp, vp, vp, vp,
                                     vp, vp, sz, vp]
    lib.spec_philox_fill.restype = i32
    lib.spec_philox_fill.argtypes = [u64, vp, i64, vp, vp]
    f32, f64 = ctypes.c_float, ctypes.c_double
    side = [vp, i32, i64, i64]  # a tensor of heads: pointer, heads, token and head strides
    lib.spec_rope_turns.restype = i32
    lib.spec_rope_turns.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp, vp]
    lib.spec_rope.restype = i32
    lib.spec_rope.argtypes = 2 * (side + [vp, i64, i64]) + [i32, i32, i64, vp, vp, i32, vp]
    lib.spec_kv_write.restype = i32
    lib.spec_kv_write.argtypes = [vp, vp, i64, i64, vp, i64, i64, i32, i64, vp, vp, vp] + side + \
        [vp, i64, i64, vp, vp]
    lib.spec_kv_read.restype = i32
    lib.spec_kv_read.argtypes = [vp, i64, vp, i32, vp, vp, vp]
    lib.spec_tree_plan_size.restype = sz
    lib.spec_tree_plan_size.argtypes = [i32]
    lib.spec_tree_plan.restype = i32
    lib.spec_tree_plan.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp,
                                   vp]
    lib.spec_tree_attention_workspace_size.restype = sz
    lib.spec_tree_attention_workspace_size.argtypes = [vp, i32]
    lib.spec_tree_attention.restype = i32
    lib.spec_tree_attention.argtypes = [vp, i64, i64, i64, i32, i32, i32, i32, vp, vp, i32, vp, vp,
                                        f32, vp, vp, vp, sz, vp, vp]
    lib.spec_kv_commit.restype = i32
    lib.spec_kv_commit.argtypes = [vp, i32, vp, vp, vp, vp, i32, i32, vp, vp, vp]
    return lib


def library_path() -> str:
    return _build.lib_path()


def lib():
    """The loaded CUDA library; raises if it has not been built."""
    global _LIB
    with _LOCK:
        if _LIB is None:
            path = _build.lib_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"spec_verify CUDA library missing ({path}); build it with "
                    "`python -m speculative_decoding_verification_51_gb300.build`")
            _LIB = _declare(ctypes.CDLL(path))
        return _LIB


def status_str(status: int) -> str:
    return lib().spec_status_str(int(status)).decode()


def workspace_size(B: int, K: int, V: int) -> int:
    return int(lib().spec_verify_workspace_size(B, K, V))


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t, name, dtype, shape=None, device=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def new_workspace(B: int, K: int, V: int, device) -> torch.Tensor:
    n = workspace_size(B, K, V)
    if n == 0:
        raise ValueError(f"unsupported sizes B={B} K={K} V={V}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def spec_verify(target_logits: torch.Tensor, draft_probs: torch.Tensor | None,
                draft_ids: torch.Tensor, num_draft: torch.Tensor, temperature: torch.Tensor,
                seed: int, *, out_ids: torch.Tensor | None = None,
                out_num_accepted: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None, request_offset: int = 0,
                debug: bool = False, dev_status: torch.Tensor | None = None,
                seed_dev: torch.Tensor | None = None, early_exit: bool = False,
                all_rows: bool = False, by_request: bool = False):
    """Verify drafts on the GPU (see include/spec_verify.h for the semantics).

    seed_dev: a one-element int64 CUDA tensor; if given, the kernels read the
    seed from it when they run (spec_verify_dev_seed, for CUDA graph capture)
    and `seed` is ignored.
    early_exit: the K + 1-pass form of reading each request's rows only up to
    its first rejection (spec_verify_early_exit); same outputs.
    all_rows: read and check every row 0..num_draft[b] in one streaming pass
    (spec_verify_all_rows); same outputs except that an all -inf sampling row
    after the first rejection makes the request bad.
    by_request: the request-by-request verifier at any B
    (spec_verify_by_request).  Without either flag the call runs the one
    verify_path() names.
    Returns (out_ids [B, K+1] int32, out_num_accepted [B] int32), plus
    (dbg_rows [B, K+1, 4], dbg_req [B, 4]) when debug=True.
    """
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, K+1, V]")
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    if target_logits.dtype == torch.bfloat16:
        dt = SPEC_BF16
    elif target_logits.dtype == torch.float32:
        dt = SPEC_F32
    else:
        raise ValueError("target_logits must be bfloat16 or float32")
    _check(target_logits, "target_logits", target_logits.dtype)
    if draft_probs is not None:
        _check(draft_probs, "draft_probs", torch.float32, (B, K, V), dev)
    _check(draft_ids, "draft_ids", torch.int32, (B, K), dev)
    _check(num_draft, "num_draft", torch.int32, (B,), dev)
    _check(temperature, "temperature", torch.float32, (B,), dev)
    if out_ids is None:
        out_ids = torch.empty((B, K1), dtype=torch.int32, device=dev)
    if out_num_accepted is None:
        out_num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    _check(out_ids, "out_ids", torch.int32, (B, K1), dev)
    _check(out_num_accepted, "out_num_accepted", torch.int32, (B,), dev)
    if workspace is None:
        workspace = new_workspace(B, K, V, dev)
    dbg_rows = dbg_req = None
    if debug:
        dbg_rows = torch.empty((B, K1, 4), dtype=torch.float32, device=dev)
        dbg_req = torch.empty((B, 4), dtype=torch.float32, device=dev)
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (1,), dev)
    if seed_dev is not None:
        _check(seed_dev, "seed_dev", torch.int64, (1,), dev)
    with torch.cuda.device(dev):
        st = _stream(stream)
        if all_rows or by_request:
            if all_rows and by_request:
                raise ValueError("all_rows and by_request exclude each other")
            fn = lib().spec_verify_all_rows if all_rows else lib().spec_verify_by_request
            rc = fn(
                _p(target_logits), dt, _p(draft_probs), _p(draft_ids), _p(num_draft),
                _p(temperature), ctypes.c_uint64(seed & (2**64 - 1)), B, K, V, _p(out_ids),
                _p(out_num_accepted), _p(workspace), workspace.numel(), st,
                ctypes.c_uint32(request_offset & 0xFFFFFFFF), _p(dbg_rows), _p(dbg_req),
                _p(dev_status), _p(seed_dev), None)
        elif early_exit:
            rc = lib().spec_verify_early_exit(
                _p(target_logits), dt, _p(draft_probs), _p(draft_ids), _p(num_draft),
                _p(temperature), ctypes.c_uint64(seed & (2**64 - 1)), B, K, V, _p(out_ids),
                _p(out_num_accepted), _p(workspace), workspace.numel(), st,
                ctypes.c_uint32(request_offset & 0xFFFFFFFF), _p(dbg_rows), _p(dbg_req),
                _p(dev_status), _p(seed_dev))
        elif seed_dev is not None:
            rc = lib().spec_verify_dev_seed(
                _p(target_logits), dt, _p(draft_probs), _p(draft_ids), _p(num_draft),
                _p(temperature), _p(seed_dev), B, K, V, _p(out_ids), _p(out_num_accepted),
                _p(workspace), workspace.numel(), st, ctypes.c_uint32(request_offset & 0xFFFFFFFF),
                _p(dbg_rows), _p(dbg_req), _p(dev_status))
        elif debug or request_offset or dev_status is not None:
            rc = lib().spec_verify_ex(
                _p(target_logits), dt, _p(draft_probs), _p(draft_ids), _p(num_draft),
                _p(temperature), ctypes.c_uint64(seed & (2**64 - 1)), B, K, V, _p(out_ids),
                _p(out_num_accepted), _p(workspace), workspace.numel(), st,
                ctypes.c_uint32(request_offset & 0xFFFFFFFF), _p(dbg_rows), _p(dbg_req),
                _p(dev_status))
        else:
            rc = lib().spec_verify(
                _p(target_logits), dt, _p(draft_probs), _p(draft_ids), _p(num_draft),
                _p(temperature), ctypes.c_uint64(seed & (2**64 - 1)), B, K, V, _p(out_ids),
                _p(out_num_accepted), _p(workspace), workspace.numel(), st)
    if rc != SPEC_OK:
        raise SpecVerifyError(rc, "spec_verify")
    if debug:
        return out_ids, out_num_accepted, dbg_rows, dbg_req
    return out_ids, out_num_accepted


def spec_verify_typical(target_logits: torch.Tensor, draft_ids: torch.Tensor,
                        num_draft: torch.Tensor, temperature: torch.Tensor, threshold: float,
                        seed: int, *, out_ids: torch.Tensor | None = None,
                        out_num_accepted: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None,
                        request_offset: int = 0, debug: bool = False,
                        dev_status: torch.Tensor | None = None):
    """Typical-acceptance verification on the GPU (include/spec_verify.h,
    spec_verify_typical): drafts are kept while p_j(x_j) >= threshold.

    Returns (out_ids, out_num_accepted), plus (dbg_rows, dbg_req) when debug=True.
    """
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, K+1, V]")
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    if target_logits.dtype == torch.bfloat16:
        dt = SPEC_BF16
    elif target_logits.dtype == torch.float32:
        dt = SPEC_F32
    else:
        raise ValueError("target_logits must be bfloat16 or float32")
    _check(target_logits, "target_logits", target_logits.dtype)
    _check(draft_ids, "draft_ids", torch.int32, (B, K), dev)
    _check(num_draft, "num_draft", torch.int32, (B,), dev)
    _check(temperature, "temperature", torch.float32, (B,), dev)
    if out_ids is None:
        out_ids = torch.empty((B, K1), dtype=torch.int32, device=dev)
    if out_num_accepted is None:
        out_num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    _check(out_ids, "out_ids", torch.int32, (B, K1), dev)
    _check(out_num_accepted, "out_num_accepted", torch.int32, (B,), dev)
    if workspace is None:
        workspace = new_workspace(B, K, V, dev)
    dbg_rows = dbg_req = None
    if debug:
        dbg_rows = torch.empty((B, K1, 4), dtype=torch.float32, device=dev)
        dbg_req = torch.empty((B, 4), dtype=torch.float32, device=dev)
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (1,), dev)
    with torch.cuda.device(dev):
        rc = lib().spec_verify_typical(
            _p(target_logits), dt, _p(draft_ids), _p(num_draft), _p(temperature),
            ctypes.c_float(threshold), ctypes.c_uint64(seed & (2**64 - 1)), B, K, V,
            _p(out_ids), _p(out_num_accepted), _p(workspace), workspace.numel(),
            _stream(stream), ctypes.c_uint32(request_offset & 0xFFFFFFFF), _p(dbg_rows),
            _p(dbg_req), _p(dev_status))
    if rc != SPEC_OK:
        raise SpecVerifyError(rc, "spec_verify_typical")
    if debug:
        return out_ids, out_num_accepted, dbg_rows, dbg_req
    return out_ids, out_num_accepted


def spec_verify_tree(target_logits: torch.Tensor, draft_probs: torch.Tensor | None,
                     tree_tokens: torch.Tensor, tree_parents: torch.Tensor,
                     num_nodes: torch.Tensor, temperature: torch.Tensor, seed: int, *,
                     workspace: torch.Tensor | None = None, stream=None, request_offset: int = 0,
                     debug: bool = False, dev_status: torch.Tensor | None = None):
    """Token-tree verification on the GPU (include/spec_verify.h,
    spec_verify_tree).  Returns (out_ids [B, N], out_num_accepted [B],
    out_last_node [B]), plus (dbg_nodes [B, N, 4], dbg_req [B, 4]) when debug."""
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, N, V]")
    B, N, V = target_logits.shape
    dev = target_logits.device
    if target_logits.dtype == torch.bfloat16:
        dt = SPEC_BF16
    elif target_logits.dtype == torch.float32:
        dt = SPEC_F32
    else:
        raise ValueError("target_logits must be bfloat16 or float32")
    _check(target_logits, "target_logits", target_logits.dtype)
    if draft_probs is not None:
        _check(draft_probs, "draft_probs", torch.float32, (B, N, V), dev)
    _check(tree_tokens, "tree_tokens", torch.int32, (B, N), dev)
    _check(tree_parents, "tree_parents", torch.int32, (B, N), dev)
    _check(num_nodes, "num_nodes", torch.int32, (B,), dev)
    _check(temperature, "temperature", torch.float32, (B,), dev)
    out_ids = torch.empty((B, N), dtype=torch.int32, device=dev)
    out_nacc = torch.empty((B,), dtype=torch.int32, device=dev)
    out_last = torch.empty((B,), dtype=torch.int32, device=dev)
    if workspace is None:
        n = int(lib().spec_verify_tree_workspace_size(B, N, V))
        if n == 0:
            raise ValueError("unsupported tree size")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    dbg_nodes = dbg_req = None
    if debug:
        dbg_nodes = torch.empty((B, N, 4), dtype=torch.float32, device=dev)
        dbg_req = torch.empty((B, 4), dtype=torch.float32, device=dev)
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (1,), dev)
    with torch.cuda.device(dev):
        rc = lib().spec_verify_tree(
            _p(target_logits), dt, _p(draft_probs), _p(tree_tokens), _p(tree_parents),
            _p(num_nodes), _p(temperature), ctypes.c_uint64(seed & (2**64 - 1)), B, N, V,
            _p(out_ids), _p(out_nacc), _p(out_last), _p(workspace), workspace.numel(),
            _stream(stream), ctypes.c_uint32(request_offset & 0xFFFFFFFF), _p(dbg_nodes),
            _p(dbg_req), _p(dev_status))
    if rc != SPEC_OK:
        raise SpecVerifyError(rc, "spec_verify_tree")
    if debug:
        return out_ids, out_nacc, out_last, dbg_nodes, dbg_req
    return out_ids, out_nacc, out_last


def spec_verify_profiled(target_logits, draft_probs, draft_ids, num_draft, temperature, seed,
                         out_ids, out_num_accepted, workspace, events, stream=None,
                         all_rows: bool = False, by_request: bool = False) -> None:
    """spec_verify (all_rows=True: spec_verify_all_rows; by_request=True:
    spec_verify_by_request) with N_MARKS torch.cuda.Event marks around its
    kernels: events[i] -> events[i + 1] brackets kernel i of KERNELS
    (KERNELS_ALL_ROWS for the all-rows verifier).  The events must already
    have been recorded once, so that they exist."""
    B, K1, V = target_logits.shape
    dt = SPEC_BF16 if target_logits.dtype == torch.bfloat16 else SPEC_F32
    if len(events) != N_MARKS:
        raise ValueError(f"need {N_MARKS} events")
    handles = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    with torch.cuda.device(target_logits.device):
        args = (_p(target_logits), dt, _p(draft_probs), _p(draft_ids), _p(num_draft),
                _p(temperature), ctypes.c_uint64(seed & (2**64 - 1)), B, K1 - 1, V, _p(out_ids),
                _p(out_num_accepted), _p(workspace), workspace.numel(), _stream(stream))
        if all_rows or by_request:
            fn = lib().spec_verify_all_rows if all_rows else lib().spec_verify_by_request
            rc = fn(*args, ctypes.c_uint32(0), None, None, None, None, handles)
        else:
            rc = lib().spec_verify_profiled(*args, handles)
    if rc != SPEC_OK:
        raise SpecVerifyError(rc, "spec_verify_profiled")


def verify_path(B: int, K: int, V: int, dtype: torch.dtype, device=None) -> int:
    """1 if spec_verify runs the request-by-request verifier for these sizes
    on `device` (default: the current CUDA device), 0 if the all-rows pass."""
    dt = SPEC_BF16 if dtype == torch.bfloat16 else SPEC_F32
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        r = lib().spec_verify_path(B, K, V, dt)
    if r < 0:
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, "spec_verify_path")
    return r


def status_word(workspace: torch.Tensor) -> torch.Tensor:
    """The device status word of the last call that used `workspace` (a view)."""
    return workspace[12:16].view(torch.int32)


def host_small_bytes(B: int, K: int) -> int:
    return int(lib().spec_verify_host_small_bytes(B, K))


def spec_verify_host(h_logits: torch.Tensor, h_probs: torch.Tensor | None, h_ids: torch.Tensor,
                     h_num: torch.Tensor, h_temp: torch.Tensor, seed: int,
                     h_out_ids: torch.Tensor, h_out_nacc: torch.Tensor, d_logits: torch.Tensor,
                     d_probs: torch.Tensor | None, d_small: torch.Tensor,
                     workspace: torch.Tensor, stream=None) -> None:
    """Host-buffer variant: copies in, verifies, copies out (asynchronous)."""
    B, K1, V = h_logits.shape
    K = K1 - 1
    dt = SPEC_BF16 if h_logits.dtype == torch.bfloat16 else SPEC_F32
    for t, n in ((h_logits, "h_logits"), (h_ids, "h_ids"), (h_num, "h_num"), (h_temp, "h_temp"),
                 (h_out_ids, "h_out_ids"), (h_out_nacc, "h_out_nacc")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous host tensor")
    with torch.cuda.device(d_logits.device):
        rc = lib().spec_verify_host(
            _p(h_logits), dt, _p(h_probs), _p(h_ids), _p(h_num), _p(h_temp),
            ctypes.c_uint64(seed & (2**64 - 1)), B, K, V, _p(h_out_ids), _p(h_out_nacc),
            _p(d_logits), _p(d_probs), _p(d_small), _p(workspace), workspace.numel(),
            _stream(stream))
    if rc != SPEC_OK:
        raise SpecVerifyError(rc, "spec_verify_host")


def philox_fill(seed: int, ctrs: torch.Tensor, stream=None) -> torch.Tensor:
    """Philox4x32-10 of the library: ctrs [n, 4] int32 (bit patterns) on the GPU."""
    _check(ctrs, "ctrs", torch.int32)
    out = torch.empty_like(ctrs)
    with torch.cuda.device(ctrs.device):
        rc = lib().spec_philox_fill(ctypes.c_uint64(seed & (2**64 - 1)), _p(ctrs),
                                    ctrs.numel() // 4, _p(out), _stream(stream))
    if rc != SPEC_OK:
        raise SpecVerifyError(rc, "spec_philox_fill")
    return out


def lmhead_logits(hidden: torch.Tensor, lm_head: torch.Tensor, *, out: torch.Tensor | None = None,
                  dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """bf16 logits = hidden [rows, H] @ lm_head [V, H]^T on the tensor cores
    (include/spec_verify.h, spec_lmhead_logits)."""
    if hidden.dim() != 2 or lm_head.dim() != 2 or hidden.shape[1] != lm_head.shape[1]:
        raise ValueError("hidden must be [rows, H] and lm_head [V, H]")
    rows, H = hidden.shape
    V = lm_head.shape[0]
    dev = hidden.device
    _check(hidden, "hidden", torch.bfloat16, device=dev)
    _check(lm_head, "lm_head", torch.bfloat16, device=dev)
    if out is None:
        out = torch.empty((rows, V), dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, (rows, V), dev)
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
    _check(dev_status, "dev_status", torch.int32, (1,), dev)
    with torch.cuda.device(dev):
        rc = lib().spec_lmhead_logits(_p(hidden), _p(lm_head), rows, H, V, _p(out), _p(dev_status),
                                      _stream(stream))
    if rc != SPEC_OK:
        raise SpecVerifyError(rc, "spec_lmhead_logits")
    return out


def spec_verify_lmhead(hidden: torch.Tensor, lm_head: torch.Tensor, draft_probs: torch.Tensor | None,
                       draft_ids: torch.Tensor, num_draft: torch.Tensor, temperature: torch.Tensor,
                       seed: int, *, logits_out: torch.Tensor | None = None,
                       out_ids: torch.Tensor | None = None,
                       out_num_accepted: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None, request_offset: int = 0,
                       debug: bool = False, dev_status: torch.Tensor | None = None):
    """Verification with the logits produced in the call from hidden states
    (include/spec_verify.h, spec_verify_lmhead).

    hidden [B, K+1, H] bf16, lm_head [V, H] bf16.  Returns (out_ids,
    out_num_accepted, logits_out) plus (dbg_rows, dbg_req) when debug=True.
    """
    if hidden.dim() != 3 or lm_head.dim() != 2 or hidden.shape[2] != lm_head.shape[1]:
        raise ValueError("hidden must be [B, K+1, H] and lm_head [V, H]")
    B, K1, H = hidden.shape
    K, V = K1 - 1, lm_head.shape[0]
    dev = hidden.device
    _check(hidden, "hidden", torch.bfloat16, device=dev)
    _check(lm_head, "lm_head", torch.bfloat16, device=dev)
    if draft_probs is not None:
        _check(draft_probs, "draft_probs", torch.float32, (B, K, V), dev)
    _check(draft_ids, "draft_ids", torch.int32, (B, K), dev)
    _check(num_draft, "num_draft", torch.int32, (B,), dev)
    _check(temperature, "temperature", torch.float32, (B,), dev)
    if logits_out is None:
        logits_out = torch.empty((B, K1, V), dtype=torch.bfloat16, device=dev)
    _check(logits_out, "logits_out", torch.bfloat16, (B, K1, V), dev)
    if out_ids is None:
        out_ids = torch.empty((B, K1), dtype=torch.int32, device=dev)
    if out_num_accepted is None:
        out_num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    _check(out_ids, "out_ids", torch.int32, (B, K1), dev)
    _check(out_num_accepted, "out_num_accepted", torch.int32, (B,), dev)
    if workspace is None:
        n = int(lib().spec_verify_lmhead_workspace_size(B, K, V, H))
        if n == 0:
            raise ValueError(f"unsupported sizes B={B} K={K} V={V} H={H}")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    dbg_rows = dbg_req = None
    if debug:
        dbg_rows = torch.empty((B, K1, 4), dtype=torch.float32, device=dev)
        dbg_req = torch.empty((B, 4), dtype=torch.float32, device=dev)
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (1,), dev)
    with torch.cuda.device(dev):
        rc = lib().spec_verify_lmhead(
            _p(hidden), _p(lm_head), H, _p(logits_out), _p(draft_probs), _p(draft_ids),
            _p(num_draft), _p(temperature), ctypes.c_uint64(seed & (2**64 - 1)), B, K, V,
            _p(out_ids), _p(out_num_accepted), _p(workspace), workspace.numel(), _stream(stream),
            ctypes.c_uint32(request_offset & 0xFFFFFFFF), _p(dbg_rows), _p(dbg_req),
            _p(dev_status))
    if rc != SPEC_OK:
        raise SpecVerifyError(rc, "spec_verify_lmhead")
    if debug:
        return out_ids, out_num_accepted, logits_out, dbg_rows, dbg_req
    return out_ids, out_num_accepted, logits_out


# ---------------------------------------------------------------- around the verification
# The pass that scores the drafted nodes, over a paged key/value cache:
# rotary positions, the cache written and read, the step's plan, the nodes'
# attention, and the kept path's rows (include/spec_verify.h).

_DTYPES = {torch.float32: SPEC_F32, torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16}
ROPE_LAYOUT = {"half": 0, "interleaved": 1}
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}


class _CCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dtype", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64)]


class _CTable(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot", ctypes.c_int), ("layout", ctypes.c_int),
                ("scale", ctypes.c_float)]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _ops():
    """The module that calls the library with torch tensors (csrc/torch_ops.cpp)."""
    global _OPS
    lib()  # raises if nothing has been built
    with _LOCK:
        if _OPS is None:
            path = _build.ops_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"spec_verify torch module missing ({path}); build it with "
                    "`python -m speculative_decoding_verification_51_gb300.build`")
            loader = importlib.machinery.ExtensionFileLoader("specverify_torch", path)
            spec = importlib.util.spec_from_file_location("specverify_torch", path, loader=loader)
            mod = importlib.util.module_from_spec(spec)
            loader.exec_module(mod)
            mod.error_class(SpecVerifyError)
            _OPS = mod
        return _OPS


def _raise(rc, what):
    if rc != SPEC_OK:
        raise SpecVerifyError(rc, what)


class RopeTable:
    """Rotary frequencies on the device (spec_rope_table)."""

    def __init__(self, turns: torch.Tensor, layout: str, scale: float):
        _check(turns, "turns", torch.int64)
        self.turns, self.rot, self.layout, self.scale = turns, 2 * turns.numel(), layout, scale
        self._c = _CTable(turns.data_ptr(), self.rot, ROPE_LAYOUT[layout], scale)
        self._ref = ctypes.addressof(self._c)


def rope_table(rot: int, *, base: float = 10000.0, layout: str = "half", scaling: str = "none",
               factor: float = 1.0, original_len: float = 0.0, fast: float = 32.0,
               slow: float = 1.0, device="cuda") -> RopeTable:
    """The frequencies of `rot` rotated channels (spec_rope_turns): `layout`
    "half" or "interleaved"; `scaling` "none", "linear", "ntk" or "by_parts"
    (which needs the original context's length; its ramp is over a pair's turns within
    that) by `factor`.  "by_parts" puts 0.1 ln(factor) + 1 on the rotated channels:
    RopeTable(t.turns, t.layout, scale) takes another."""
    if layout not in ROPE_LAYOUT:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUT)}")
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALING)}")
    turns = torch.empty(max(int(rot) // 2, 1), dtype=torch.int64)
    scale = ctypes.c_float()
    _raise(lib().spec_rope_turns(rot, base, ROPE_SCALING[scaling], factor, original_len, fast,
                                 slow, turns.data_ptr(), ctypes.addressof(scale)),
           "spec_rope_turns")
    return RopeTable(turns.to(device), layout, scale.value)


def rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, table: RopeTable, *,
         out_q: torch.Tensor | None = None, out_k: torch.Tensor | None = None,
         inverse: bool = False, stream=None):
    """Rotary positions (spec_rope): q [..., q_heads, D] and k [..., k_heads,
    D] (or None) turned by positions [tokens] int32.  out_q / out_k: new
    tensors, or given ones (q and k themselves: in place).  inverse=True is the
    transpose, which takes gradients of the outputs to gradients of the inputs: it
    turns by the negative angles with the table's factor on the rotated channels
    (1 but for "by_parts"), so that it is the inverse where that is 1.
    Returns (out_q, out_k), or out_q where k is None."""
    return (_OPS or _ops()).rope(q, k, positions, table, out_q, out_k, inverse, stream)


class KVCache:
    """A paged key/value cache of one layer (spec_kv_cache): k and v
    [num_pages, heads, page_size, head_dim] (bfloat16, float16, or uint8 /
    float8_e4m3fn with k_scale and v_scale [num_pages, heads, page_size]
    uint8).  Any strides with contiguous channels, the same for k and v: a
    [num_pages, page_size, heads, head_dim] allocation is passed as its
    transpose(1, 2).  The tensors stay the caller's."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must be [num_pages, heads, page_size, head_dim], alike")
        if k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must have equal strides and contiguous channels")
        if not k.is_cuda:
            raise ValueError("the cache must be CUDA tensors")
        P, H, S, D = k.shape
        if k.dtype in (torch.uint8, torch.float8_e4m3fn):
            dt = SPEC_E4M3
            if k_scale is None or v_scale is None:
                raise ValueError("an 8-bit cache needs k_scale and v_scale")
            for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                _check(t, n, torch.uint8, (P, H, S), k.device)
        elif k.dtype in (torch.bfloat16, torch.float16):
            dt = _DTYPES[k.dtype]
            if k_scale is not None or v_scale is not None:
                raise ValueError("a 16-bit cache has no scales")
        else:
            raise ValueError(f"a cache of {k.dtype} is not supported")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.heads, self.page_size, self.head_dim = P, H, S, D
        self.device, self.dtype = k.device, dt
        self._c = _CCache(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale), dt, P, S, H, D,
                          k.stride(0), k.stride(1), k.stride(2))
        self._ref = ctypes.addressof(self._c)


def new_kv_cache(num_pages: int, page_size: int, heads: int, head_dim: int, *,
                 dtype=torch.bfloat16, device="cuda") -> KVCache:
    """A cache of its own memory; dtype bfloat16, float16 or float8_e4m3fn."""
    shape = (num_pages, heads, page_size, head_dim)
    if dtype == torch.float8_e4m3fn:
        dtype = torch.uint8
    k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    sc = (None, None)
    if dtype == torch.uint8:
        sc = tuple(torch.full(shape[:3], 127, dtype=torch.uint8, device=device) for _ in range(2))
    return KVCache(k, v, *sc)


def kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, *,
             positions: torch.Tensor | None = None, table: RopeTable | None = None,
             q: torch.Tensor | None = None, out_q: torch.Tensor | None = None,
             dev_status: torch.Tensor | None = None, stream=None):
    """Write key and value rows [..., heads, head_dim] to their cache slots
    (spec_kv_write); slots [tokens] int64, negative: not written.  With
    `table` and `positions` the keys are rotated on the way, and q [...,
    q_heads, head_dim] into out_q (a new tensor by default), which is
    returned."""
    return (_OPS or _ops()).kv_write(cache, k, v, slots, positions, table, q, out_q, dev_status, stream)


def kv_read(cache: KVCache, slots: torch.Tensor, *, dtype: torch.dtype | None = None,
            out_k: torch.Tensor | None = None, out_v: torch.Tensor | None = None, stream=None):
    """The rows of `slots` (int64, any shape) as (k, v) [*slots.shape, heads,
    head_dim] of `dtype` (the cache's own by default, bfloat16 for an 8-bit
    one); a slot outside the cache reads as zeros (spec_kv_read)."""
    return (_OPS or _ops()).kv_read(cache, slots, dtype, out_k, out_v, stream)


@dataclass
class TreePlan:
    """Where the nodes of a step stand (spec_tree_plan).  One plan serves every
    layer of the step, on any number of streams."""
    positions: torch.Tensor    # [B, N] int32
    slots: torch.Tensor        # [B, N] int64
    masks: torch.Tensor        # [B, N] int32: bit u: node u is this one or above it
    context_len: torch.Tensor  # [B] int32 (the caller's)
    page_table: torch.Tensor   # [B, max_pages] int32 (the caller's)
    page_size: int
    num_pages: int
    buffer: torch.Tensor       # the division of the attention's work
    workspace: dict            # of tree_attention, by (stream, heads, head_dim)


def tree_plan(tree_parents: torch.Tensor, num_nodes: torch.Tensor, context_len: torch.Tensor,
              page_table: torch.Tensor, cache: KVCache, *, dev_status: torch.Tensor | None = None,
              stream=None) -> TreePlan:
    """Positions, cache slots and ancestor masks of the nodes [B, N] that
    follow each request's context (spec_tree_plan); `cache` gives the pages'
    size and number."""
    positions, slots, masks, buffer = (_OPS or _ops()).tree_plan(
        tree_parents, num_nodes, context_len, page_table, cache, dev_status, stream)
    return TreePlan(positions, slots, masks, context_len, page_table, cache.page_size,
                    cache.num_pages, buffer, {})


def tree_attention(q: torch.Tensor, cache: KVCache, plan: TreePlan, *, scale: float | None = None,
                   masks: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of the nodes' queries q [B, N, q_heads, head_dim] over the
    cache (spec_tree_attention).  scale: 1 / sqrt(head_dim) by default; masks
    [B, N] int32: the plan's by default; lse [B, N, q_heads] float32: written
    where given.  The workspace is kept with the plan unless one is given."""
    return (_OPS or _ops()).tree_attention(q, cache, plan, scale, masks, out, lse, workspace, dev_status,
                                           stream)


def kv_commit(caches: list, plan: TreePlan, last_node: torch.Tensor, *,
              new_context_len: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """After the verification: move the kept path's rows to the places after
    the context in every cache of `caches` (the layers) and return the new
    context lengths (spec_kv_commit).  last_node: spec_verify_tree's third
    result, or spec_verify's second for a chain.  new_context_len may be the
    plan's context_len itself."""
    return (_OPS or _ops()).kv_commit(caches, plan, last_node, new_context_len, dev_status, stream)
