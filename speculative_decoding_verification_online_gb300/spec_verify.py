"""ctypes binding of the CUDA verifier library (``libspec_verify.so``).

Argument marshalling only: every step of the verification runs in the CUDA
kernels behind the C ABI of ``include/spec_verify.h``.  Functions keep the C
names; ``SpecVerifier`` bundles a handle with torch-tensor marshalling
(``data_ptr()`` and the current CUDA stream).  ``stream=`` runs a call on
another stream (a raw handle or a ``torch.cuda.Stream``); the results that it
makes are then memory of that stream, and the caller orders the streams around
the inputs and the results.  There is no CPU fallback: if the shared library is
missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libspec_verify.so")

SV_OK, SV_EINVAL, SV_ENOMEM, SV_ECUDA, SV_EUNSUPPORTED = 0, 1, 2, 3, 4
SV_F32, SV_BF16 = 0, 1
SV_PLAIN, SV_GATED_MU = 0, 1
SV_FLAG_UNREACHED, SV_FLAG_ACCEPT, SV_FLAG_REJECT, SV_FLAG_NULL, SV_FLAG_INVALID = 0, 1, 2, 3, 4
(SV_CNT_TESTED, SV_CNT_ACCEPTED, SV_CNT_NULL, SV_CNT_REJECTED, SV_CNT_BONUS, SV_CNT_BOUNDARY, SV_CNT_INVALID,
 SV_CNT_DEGENERATE) = range(8)
COUNTER_NAMES = ("tested", "accepted", "null", "rejected", "bonus", "boundary", "invalid",
                 "degenerate")
SV_MAX_K = 32
SV_MAX_V = 1 << 22
SV_MAX_NODES = 256
(SV_ACT_NONE, SV_ACT_RELU, SV_ACT_SILU, SV_ACT_GELU, SV_ACT_GELU_TANH, SV_ACT_SOFTCAP) = range(6)
ACTIVATIONS = {"none": SV_ACT_NONE, "relu": SV_ACT_RELU, "silu": SV_ACT_SILU, "gelu": SV_ACT_GELU,
               "gelu_tanh": SV_ACT_GELU_TANH, "softcap": SV_ACT_SOFTCAP}
SV_WITH_REPLACEMENT, SV_WITHOUT_REPLACEMENT = 0, 1
RUN_HIDDEN_PENALTIES = frozenset(("history", "history_len", "prompt_len", "repetition", "frequency", "presence", "bias", "mask",
                                  "mask_row", "draft_mask", "draft_mask_row"))

_lib = None


class SpecVerifyError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {spec_verify_status_string(status)} (status {status})")


def load() -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY):
        raise RuntimeError(f"CUDA library {LIBRARY} is not built; run __graft_entry__.build()")
    L = ctypes.CDLL(LIBRARY)
    P, I, F, U64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_uint64
    L.spec_verify_init.argtypes = [ctypes.POINTER(P), I, I, I, I]
    L.spec_verify_init.restype = I
    run_common = [P, P, I, P, I, P, I, F, I, F, P, P, U64]
    L.spec_verify_run.argtypes = run_common + [P, P, P, P, P, P]
    L.spec_verify_run.restype = I
    L.spec_verify_run_ex.argtypes = run_common + [U64, P, P, P, P, P, P, P, P, P]
    L.spec_verify_run_ex.restype = I
    L.spec_verify_run_host.argtypes = run_common + [P, P, P, P, P, P]
    L.spec_verify_run_host.restype = I
    L.spec_verify_free.argtypes = [P]
    L.spec_verify_free.restype = I
    L.spec_verify_status_string.argtypes = [I]
    L.spec_verify_status_string.restype = ctypes.c_char_p
    L.spec_verify_launches_per_run.argtypes = []
    L.spec_verify_launches_per_run.restype = I
    L.spec_verify_mark_next.argtypes = [P, P, P]
    L.spec_verify_mark_next.restype = I
    L.spec_verify_run_noalloc.argtypes = [P, I, P, I, P, I, I, I, F, I, F, P, P, U64, P, P, P, P, P, P]
    L.spec_verify_run_noalloc.restype = I
    L.spec_verify_set_gate_policy.argtypes = [P, P, I, F]
    L.spec_verify_set_gate_policy.restype = I
    L.spec_verify_diagnostics.argtypes = [P, P, I, P, I, P, I, F, I, F, P, P, P, P, P, P]
    L.spec_verify_diagnostics.restype = I
    L.spec_verify_set_filters.argtypes = [P, I, F, F, I, F, F]
    L.spec_verify_set_filters.restype = I
    L.spec_verify_launches_per_filtered_run.argtypes = []
    L.spec_verify_launches_per_filtered_run.restype = I
    I64 = ctypes.c_int64
    L.spec_verify_linear.argtypes = [P, I64, I64, P, I64, I64, P, I, I64, P, I, I64, I64, P, I, I64, I64, I, I, I, I, I,
                                     F, I, P]
    L.spec_verify_linear.restype = I
    L.spec_verify_softmax.argtypes = [P, I, I64, I, I, F, P, P, I64, I, P]
    L.spec_verify_softmax.restype = I
    L.spec_verify_tree.argtypes = [P, I64, P, I64, I, P, P, P, P, P, P, I, I, I, I, I, I, P, P, P, P, P, P, I, P]
    L.spec_verify_tree.restype = I
    L.spec_verify_penalties.argtypes = [P, I, I64, P, I, I64, I, P, I64, I, P, P, P, P, P, I, I, I, P, P, P, P, P, P, I, P,
                                        I64, I, P, I, P]
    L.spec_verify_penalties.restype = I
    L.spec_verify_cache_write.argtypes = [P, P, P, I, I64, I64, I64, I64, P, I64, I, P, P, I, I, I, I, P]
    L.spec_verify_cache_write.restype = I
    L.spec_verify_cache_keep.argtypes = [P, P, I, P, P, I64, I, P, P, I, I, P]
    L.spec_verify_cache_keep.restype = I
    L.spec_verify_attend_workspace.argtypes = [I, I, I, I, I]
    L.spec_verify_attend_workspace.restype = ctypes.c_size_t
    L.spec_verify_attend.argtypes = [P, P, I64, I64, P, I64, I64, I, F, P, I64, I, P, P, P, I, I, I, P, ctypes.c_size_t, I,
                                     P]
    L.spec_verify_attend.restype = I
    _lib = L
    return L


# ------------------------------------------------------------- C names

def spec_verify_status_string(status: int) -> str:
    return load().spec_verify_status_string(int(status)).decode()


def spec_verify_init(max_B: int, k: int, V: int, device: int = 0) -> int:
    h = ctypes.c_void_p()
    rc = load().spec_verify_init(ctypes.byref(h), int(max_B), int(k), int(V), int(device))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_init")
    return h.value


def spec_verify_run(h, Lt, tdt, Ld, ddt, D, B, temperature, gate_mode, threshold, gate_per_seq,
                    threshold_per_seq, seed, accepted_len, tokens, accept_prob, flags, counters,
                    stream) -> int:
    """Raw call with integer pointers; returns the status code."""
    return load().spec_verify_run(h, Lt, tdt, Ld, ddt, D, B, temperature, gate_mode, threshold,
                                  gate_per_seq, threshold_per_seq, seed, accepted_len, tokens,
                                  accept_prob, flags, counters, stream)


def spec_verify_run_ex(h, Lt, tdt, Ld, ddt, D, B, temperature, gate_mode, threshold, gate_per_seq,
                       threshold_per_seq, seed, seq_offset, u_accept, u_residual, accepted_len,
                       tokens, accept_prob, flags, counters, row_stats, stream) -> int:
    return load().spec_verify_run_ex(h, Lt, tdt, Ld, ddt, D, B, temperature, gate_mode, threshold,
                                     gate_per_seq, threshold_per_seq, seed, seq_offset, u_accept,
                                     u_residual, accepted_len, tokens, accept_prob, flags, counters,
                                     row_stats, stream)


def spec_verify_run_host(h, Lt, tdt, Ld, ddt, D, B, temperature, gate_mode, threshold,
                         gate_per_seq, threshold_per_seq, seed, accepted_len, tokens, accept_prob,
                         flags, counters, stream) -> int:
    return load().spec_verify_run_host(h, Lt, tdt, Ld, ddt, D, B, temperature, gate_mode,
                                       threshold, gate_per_seq, threshold_per_seq, seed,
                                       accepted_len, tokens, accept_prob, flags, counters, stream)


def spec_verify_free(h) -> int:
    return load().spec_verify_free(h)


def spec_verify_set_gate_policy(h, schedule, n_schedule, min_cum) -> int:
    """Raw call: schedule is a ctypes float array (or None), min_cum a float."""
    return load().spec_verify_set_gate_policy(h, schedule, n_schedule, min_cum)


def spec_verify_diagnostics(h, Lt, tdt, Ld, ddt, D, B, temperature, gate_mode, threshold,
                            gate_per_seq, threshold_per_seq, min_sum, pq_sum, argmax_q, stream) -> int:
    """Raw call of the acceptance diagnostics; returns the status."""
    return load().spec_verify_diagnostics(h, Lt, tdt, Ld, ddt, D, B, temperature, gate_mode,
                                          threshold, gate_per_seq, threshold_per_seq, min_sum,
                                          pq_sum, argmax_q, stream)


def spec_verify_set_filters(h, top_k_t, top_p_t, min_p_t, top_k_d, top_p_d, min_p_d) -> int:
    """Raw call: sampler filters of the target and draft rows."""
    return load().spec_verify_set_filters(h, top_k_t, top_p_t, min_p_t, top_k_d, top_p_d, min_p_d)


def spec_verify_launches_per_filtered_run() -> int:
    return load().spec_verify_launches_per_filtered_run()


def spec_verify_launches_per_run() -> int:
    return load().spec_verify_launches_per_run()


def spec_verify_mark_next(h, ev_before, ev_after) -> int:
    """Record two CUDA events (raw cudaEvent_t handles) around the next call's stream pass."""
    return load().spec_verify_mark_next(h, ev_before, ev_after)


def spec_verify_run_noalloc(Lt, tdt, Ld, ddt, D, B, k, V, temperature, gate_mode, threshold,
                            gate_per_seq, threshold_per_seq, seed, accepted_len, tokens, accept_prob,
                            flags, counters, stream) -> int:
    """Raw call of the allocation-free entry point (current device); returns the status."""
    return load().spec_verify_run_noalloc(Lt, tdt, Ld, ddt, D, B, k, V, temperature, gate_mode,
                                          threshold, gate_per_seq, threshold_per_seq, seed,
                                          accepted_len, tokens, accept_prob, flags, counters,
                                          stream)


def spec_verify_linear(x, x_row, x_group, w, w_row, w_group, bias, bias_dt, bias_group, residual, residual_dt,
                       residual_row, residual_group, y, y_dt, y_row, y_group, groups, M, N, K, act, cap, device,
                       stream) -> int:
    """Raw call of the grouped matrix product; returns the status."""
    return load().spec_verify_linear(x, x_row, x_group, w, w_row, w_group, bias, bias_dt, bias_group, residual,
                                     residual_dt, residual_row, residual_group, y, y_dt, y_row, y_group, groups, M, N,
                                     K, act, cap, device, stream)


def spec_verify_softmax(logits, dt, logits_stride, rows, V, temperature, temperature_per_row, probs, probs_stride,
                        device, stream) -> int:
    """Raw call of the logits rows' probabilities; returns the status."""
    return load().spec_verify_softmax(logits, dt, logits_stride, rows, V, temperature, temperature_per_row, probs,
                                      probs_stride, device, stream)


def spec_verify_tree(p, p_stride, q, q_stride, draft_rows, node_start, tokens, parent, draft_row, u_accept, u_pick, B,
                     total_nodes, max_nodes, max_depth, V, siblings, accepted_len, out_tokens, path, accept_prob,
                     flags, counters, device, stream) -> int:
    """Raw call of the tree verification; returns the status."""
    return load().spec_verify_tree(p, p_stride, q, q_stride, draft_rows, node_start, tokens, parent, draft_row,
                                   u_accept, u_pick, B, total_nodes, max_nodes, max_depth, V, siblings, accepted_len,
                                   out_tokens, path, accept_prob, flags, counters, device, stream)


class SvCache(ctypes.Structure):
    """sv_cache of include/spec_verify.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("scale_layer_stride", ctypes.c_int64), ("layers", ctypes.c_int),
                ("pages", ctypes.c_int), ("heads", ctypes.c_int), ("page_tokens", ctypes.c_int), ("block", ctypes.c_int),
                ("dim", ctypes.c_int)]


def spec_verify_penalties(logits, dt, logits_stride, out, out_dt, out_stride, V, history, history_stride, history_cap,
                          history_len, prompt_len, node_tokens, parent, node_start, B, total_nodes, max_nodes, repetition,
                          frequency, presence, bias_start, bias_tokens, bias_values, total_biases, mask, mask_stride,
                          mask_rows, mask_row, device, stream) -> int:
    """Raw call of the penalties, biases and masks on logits rows; returns the status."""
    return load().spec_verify_penalties(logits, dt, logits_stride, out, out_dt, out_stride, V, history, history_stride,
                                        history_cap, history_len, prompt_len, node_tokens, parent, node_start, B,
                                        total_nodes, max_nodes, repetition, frequency, presence, bias_start, bias_tokens,
                                        bias_values, total_biases, mask, mask_stride, mask_rows, mask_row, device, stream)


def spec_verify_cache_write(cache, k, v, dt, k_row, k_head, v_row, v_head, page_table, table_stride, table_cols, context,
                            node_start, B, total_nodes, max_nodes, device, stream) -> int:
    """Raw call that writes a step's rows into a cache (a pointer to SvCache); returns the status."""
    return load().spec_verify_cache_write(cache, k, v, dt, k_row, k_head, v_row, v_head, page_table, table_stride,
                                          table_cols, context, node_start, B, total_nodes, max_nodes, device, stream)


def spec_verify_cache_keep(cache, path, max_depth, accepted_len, page_table, table_stride, table_cols, context, new_context,
                           B, device, stream) -> int:
    """Raw call that keeps the rows of the accepted paths; returns the status."""
    return load().spec_verify_cache_keep(cache, path, max_depth, accepted_len, page_table, table_stride, table_cols, context,
                                         new_context, B, device, stream)


def spec_verify_attend_workspace(heads, q_heads, dim, max_nodes, device) -> int:
    """Bytes of workspace of an attention call."""
    return load().spec_verify_attend_workspace(heads, q_heads, dim, max_nodes, device)


def spec_verify_attend(cache, q, q_row, q_head, out, out_row, out_head, q_heads, scale, page_table, table_stride, table_cols,
                       context, node_start, parent, B, total_nodes, max_nodes, workspace, workspace_bytes, device,
                       stream) -> int:
    """Raw call of a step's attention over a cache; returns the status."""
    return load().spec_verify_attend(cache, q, q_row, q_head, out, out_row, out_head, q_heads, scale, page_table,
                                     table_stride, table_cols, context, node_start, parent, B, total_nodes, max_nodes,
                                     workspace, workspace_bytes, device, stream)


# ------------------------------------------------------ torch marshalling

def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float32:
        return SV_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(t: torch.Tensor, name: str, shape, dtype=None, device=None):
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype} != {dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_rows(t: torch.Tensor, name: str, dim: int, dtype=None, device=None):
    """A tensor of ``dim`` dimensions whose rows are contiguous, the other strides being free; returns its strides."""
    strides = t.stride()
    if len(strides) != dim:
        raise ValueError(f"{name}: {len(strides)} dimensions, expected {dim}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype} != {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if strides[-1] != 1 and t.shape[-1] > 1 and 0 not in t.shape:
        raise ValueError(f"{name}: rows must be contiguous")
    return strides


def _cuda_device(t: torch.Tensor, name: str):
    if t.device.type != "cuda":
        raise ValueError(f"{name}: on {t.device}, expected a CUDA device")
    return t.device


def _stream(dev: torch.device, stream):
    # the handle of current_stream(dev) without its Python object: 0.1 us against 2 us
    return torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream


def _new(dev: torch.device, stream, make):
    """The results that ``make`` allocates, as memory of the stream that the call runs on: torch gives a tensor's memory
    on in the order of the stream it was allocated under, and a call on another one stands outside of that order."""
    if stream is None:
        return make()
    if not isinstance(stream, torch.cuda.Stream):
        handle = getattr(stream, "value", stream) or 0
        if handle == torch._C._cuda_getCurrentRawStream(dev.index):
            return make()
        # (an ExternalStream of handle 0 would be a new stream)
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return make()


def linear(x, weight, bias=None, residual=None, activation="none", cap=0.0, out=None, out_dtype=None, stream=None):
    """act(x @ weight.T + bias) + residual, with the sums and the epilogue in fp32 and one rounding.

    ``x`` [M, K] and ``weight`` [N, K] give [M, N]; ``weight`` [G, N, K] (one
    matrix per head) with ``x`` [G, M, K], or [M, K] shared by the heads, gives
    [G, M, N].  ``x`` and ``weight`` are bfloat16; ``bias`` [N] / [G, N],
    ``residual`` and ``out`` (shaped as the result) bfloat16 or float32.  Only
    rows have to be contiguous: ``out=logits.transpose(0, 1)`` writes heads
    straight into [M, G, N].  ``activation``: none, relu, silu, gelu, gelu_tanh,
    or softcap (``cap`` * tanh(z / ``cap``)).  ``out`` may be ``residual``
    itself, but share no memory with ``x``, ``weight`` and ``bias``.  A new result takes ``out_dtype`` (default bfloat16).  No gradient
    is recorded."""
    dev = _cuda_device(x, "x")
    bf16 = torch.bfloat16
    wshape, xshape = weight.shape, x.shape
    dim = len(wshape)
    if dim not in (2, 3):
        raise ValueError(f"weight: {dim} dimensions, expected 2 or 3")
    ws = _check_rows(weight, "weight", dim, bf16, dev)
    grouped = dim == 3
    shared = len(xshape) == 2
    xs = _check_rows(x, "x", 2 if shared else 3, bf16, dev)
    G = wshape[0] if grouped else 1
    if not shared and (not grouped or xshape[0] != G):
        raise ValueError(f"x: shape {tuple(xshape)} does not go with weight {tuple(wshape)}")
    M, N, K = xshape[-2], wshape[-2], wshape[-1]
    if xshape[-1] != K:
        raise ValueError(f"x: rows of {xshape[-1]}, weight has rows of {K}")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation {activation!r} is not one of {sorted(ACTIVATIONS)}")
    shape = (G, M, N) if grouped else (M, N)
    if out is None:
        out = _new(dev, stream, lambda: torch.empty(shape, dtype=out_dtype or bf16, device=dev))
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out: dtype {out.dtype} != {out_dtype}")
    ys = _check_rows(out, "out", dim, None, dev)
    if out.shape != shape:
        raise ValueError(f"out: shape {tuple(out.shape)} != {shape}")
    rp, rdt, rrow, rgroup = None, 0, 0, 0
    if residual is not None:
        rs = _check_rows(residual, "residual", dim, None, dev)
        if residual.shape != shape:
            raise ValueError(f"residual: shape {tuple(residual.shape)} != {shape}")
        rp, rdt, rrow, rgroup = residual.data_ptr(), _dt(residual), rs[-2], rs[0] if grouped else 0
    bp, bdt, bgroup = None, 0, 0
    if bias is not None:
        bs = _check_rows(bias, "bias", dim - 1, None, dev)
        if bias.shape != ((G, N) if grouped else (N,)):
            raise ValueError(f"bias: shape {tuple(bias.shape)} != {(G, N) if grouped else (N,)}")
        bp, bdt, bgroup = bias.data_ptr(), _dt(bias), bs[0] if grouped else 0
    rc = spec_verify_linear(
        x.data_ptr(), xs[-2], 0 if shared else xs[0], weight.data_ptr(), ws[-2], ws[0] if grouped else 0, bp, bdt, bgroup,
        rp, rdt, rrow, rgroup, out.data_ptr(), _dt(out), ys[-2], ys[0] if grouped else 0, G, M, N, K, act, float(cap),
        dev.index, _stream(dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_linear")
    return out


def softmax(logits, temperature, out=None, stream=None):
    """Probabilities of logits rows [rows, V] (bfloat16 or float32, rows contiguous) as fp32 [rows, V].

    ``temperature``: a float, or a float32 tensor [rows] on the device; 0 puts 1
    on a row's first largest logit.  Rows without a distribution (a NaN or +inf
    logit, every logit -inf, a bad temperature of their own) become NaN."""
    dev = _cuda_device(logits, "logits")
    _check_rows(logits, "logits", 2, None, dev)
    rows, V = logits.shape
    per_row = None
    if isinstance(temperature, torch.Tensor):
        _check(temperature, "temperature", (rows,), torch.float32, dev)
        per_row, temperature = temperature.data_ptr(), 1.0
    if out is None:
        out = _new(dev, stream, lambda: torch.empty(rows, V, dtype=torch.float32, device=dev))
    else:
        _check_rows(out, "out", 2, torch.float32, dev)
        if out.shape != logits.shape:
            raise ValueError(f"out: shape {tuple(out.shape)} != {tuple(logits.shape)}")
    rc = spec_verify_softmax(logits.data_ptr(), _dt(logits), logits.stride(0), rows, V, float(temperature), per_row,
                             out.data_ptr(), out.stride(0), dev.index, _stream(dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_softmax")
    return out


def verify_tree(target_probs, draft_probs, tokens, parent, draft_row, node_start, u_accept, u_pick, max_nodes=None,
                max_depth=None, replacement=True, counters=None, out=None, stream=None):
    """Verify drafted trees (ragged batches, several candidates per place) from probabilities and given uniforms.

    ``node_start`` [B + 1], ``tokens``, ``parent`` [nodes] and ``draft_row``
    [nodes + B] are int32, ``u_accept`` [nodes] and ``u_pick`` [B] float32;
    ``target_probs`` [nodes + B, V] holds each sequence's root row, then its
    nodes' rows; ``draft_probs`` [draft rows, V] (or None) the distributions
    that ``draft_row`` names, -1 for certain proposals (see
    ``spec_verify_tree`` in include/spec_verify.h).  ``max_nodes`` and
    ``max_depth`` bound a sequence's nodes and its depth (default: the number
    of nodes, as far as SV_MAX_NODES).  ``replacement``: whether siblings were
    drawn with replacement.  Returns accepted_len [B], tokens [B, max_depth + 1],
    path [B, max_depth], accept_prob and flags [nodes]."""
    dev = _cuda_device(target_probs, "target_probs")
    f32, i32 = torch.float32, torch.int32
    p_stride = _check_rows(target_probs, "target_probs", 2, f32, dev)[0]
    rows_p, V = target_probs.shape
    B, total = u_pick.shape[0], tokens.shape[0]
    if rows_p != total + B:
        raise ValueError(f"target_probs: {rows_p} rows, expected {total + B}")
    q, rows_q, q_stride = None, 0, 0
    if draft_probs is not None:
        q_stride = _check_rows(draft_probs, "draft_probs", 2, f32, dev)[0]
        q, (rows_q, V_q) = draft_probs.data_ptr(), draft_probs.shape
        if V_q != V:
            raise ValueError(f"draft_probs: rows of {V_q}, expected {V}")
    nodes = (total,)
    _check(tokens, "tokens", nodes, i32, dev)
    _check(parent, "parent", nodes, i32, dev)
    _check(draft_row, "draft_row", (total + B,), i32, dev)
    _check(node_start, "node_start", (B + 1,), i32, dev)
    _check(u_accept, "u_accept", nodes, f32, dev)
    _check(u_pick, "u_pick", (B,), f32, dev)
    if counters is not None:
        _check(counters, "counters", (8,), torch.int64, dev)
    if max_nodes is None:
        max_nodes = min(total, SV_MAX_NODES)
    if max_depth is None:
        max_depth = max_nodes
    if out is None:
        out = _new(dev, stream, lambda: dict(
            accepted_len=torch.empty(B, dtype=i32, device=dev),
            tokens=torch.empty(B, max_depth + 1, dtype=i32, device=dev),
            path=torch.empty(B, max_depth, dtype=i32, device=dev),
            accept_prob=torch.empty(total, dtype=f32, device=dev),
            flags=torch.empty(total, dtype=torch.int8, device=dev)))
    else:
        for name, shp, dtype in (("accepted_len", (B,), i32), ("tokens", (B, max_depth + 1), i32),
                                 ("path", (B, max_depth), i32), ("accept_prob", (total,), f32),
                                 ("flags", (total,), torch.int8)):
            if name in out:
                _check(out[name], name, shp, dtype, dev)
    rc = spec_verify_tree(
        target_probs.data_ptr(), p_stride, q, q_stride, rows_q, node_start.data_ptr(),
        tokens.data_ptr(), parent.data_ptr(), draft_row.data_ptr(), u_accept.data_ptr(), u_pick.data_ptr(), B, total,
        max_nodes, max_depth, V, SV_WITH_REPLACEMENT if replacement else SV_WITHOUT_REPLACEMENT,
        out["accepted_len"].data_ptr(), out["tokens"].data_ptr(), _ptr(out.get("path")), _ptr(out.get("accept_prob")),
        _ptr(out.get("flags")), _ptr(counters), dev.index, _stream(dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_tree")
    return out


def penalize(logits, history, history_len, tokens, parent, node_start, prompt_len=None, repetition=None, frequency=None,
             presence=None, bias=None, mask=None, mask_row=None, max_nodes=None, out=None, stream=None):
    """Penalties for repeated tokens, biases and masks on logits rows, as ``spec_verify_penalties`` has them.

    ``logits`` [nodes + B, V] (bfloat16 or float32, rows contiguous) holds each
    sequence's root row, then its nodes' rows, as ``verify_tree`` takes them; a
    row counts the tokens of ``history`` [B, cap] (int32; ``history_len`` [B] of
    them, the first ``prompt_len`` [B] for ``repetition`` only) and of its own
    path: ``tokens``, ``parent`` [nodes] (None: chains), ``node_start`` [B + 1].
    ``repetition``, ``frequency``, ``presence``: float32 [B] or None.  ``bias``:
    (start [B + 1], tokens, values) with int32, int32 and float32 entries.
    ``mask`` [masks, >= V / 32] int32, a bit for each allowed token, for the row
    itself or the one that ``mask_row`` [nodes + B] names (-1: none).  ``out``: the
    results' tensor, may be ``logits`` (then only what changes is written);
    default: a new one of the same type."""
    dev = _cuda_device(logits, "logits")
    i32, f32 = torch.int32, torch.float32
    x_stride = _check_rows(logits, "logits", 2, None, dev)[0]
    rows, V = logits.shape
    B, total = history_len.shape[0], tokens.shape[0]
    if rows != total + B:
        raise ValueError(f"logits: {rows} rows, expected {total + B}")
    h_stride = _check_rows(history, "history", 2, i32, dev)[0]
    if history.shape[0] != B:
        raise ValueError(f"history: {history.shape[0]} rows, expected {B}")
    _check(history_len, "history_len", (B,), i32, dev)
    _check(tokens, "tokens", (total,), i32, dev)
    _check(node_start, "node_start", (B + 1,), i32, dev)
    if parent is not None:
        _check(parent, "parent", (total,), i32, dev)
    if prompt_len is not None:
        _check(prompt_len, "prompt_len", (B,), i32, dev)
    for name, t in (("repetition", repetition), ("frequency", frequency), ("presence", presence)):
        if t is not None:
            _check(t, name, (B,), f32, dev)
    b_start = b_tokens = b_values = None
    biases = 0
    if bias is not None:
        start, b_t, b_v = bias
        biases = b_t.shape[0]
        _check(start, "bias start", (B + 1,), i32, dev)
        _check(b_t, "bias tokens", (biases,), i32, dev)
        _check(b_v, "bias values", (biases,), f32, dev)
        b_start, b_tokens, b_values = start.data_ptr(), b_t.data_ptr(), b_v.data_ptr()
    m_ptr, m_stride, m_rows = None, 0, 0
    if mask is not None:
        m_stride = _check_rows(mask, "mask", 2, i32, dev)[0]
        m_rows = mask.shape[0]
        if mask.shape[1] < (V + 31) // 32:
            raise ValueError(f"mask: rows of {mask.shape[1]} words, expected {(V + 31) // 32}")
        if mask_row is None and m_rows != rows:
            raise ValueError(f"mask: {m_rows} rows, expected {rows}")
        m_ptr = mask.data_ptr()
        if mask_row is not None:
            _check(mask_row, "mask_row", (rows,), i32, dev)
    elif mask_row is not None:
        raise ValueError("mask_row: there is no mask")
    if max_nodes is None:
        max_nodes = min(total, SV_MAX_NODES)
    if out is None:
        out = _new(dev, stream, lambda: torch.empty(rows, V, dtype=logits.dtype, device=dev))
    y_stride = _check_rows(out, "out", 2, None, dev)[0]
    if out.shape != logits.shape:
        raise ValueError(f"out: shape {tuple(out.shape)} != {tuple(logits.shape)}")
    rc = spec_verify_penalties(
        logits.data_ptr(), _dt(logits), x_stride, out.data_ptr(), _dt(out), y_stride, V, history.data_ptr(), h_stride,
        history.shape[1], history_len.data_ptr(), _ptr(prompt_len), tokens.data_ptr(), _ptr(parent), node_start.data_ptr(),
        B, total, max_nodes, _ptr(repetition), _ptr(frequency), _ptr(presence), b_start, b_tokens, b_values, biases, m_ptr,
        m_stride, m_rows, _ptr(mask_row), dev.index, _stream(dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_penalties")
    return out


class PagedCache(NamedTuple):
    """Keys and values in pages of 8-bit entries, with a scale for each block of tokens and head.

    ``k``, ``v``: float8_e4m3fn [pages, heads, page tokens, dim], or with the
    layers of a model in front; only the entries of a token have to be
    contiguous, so that either of heads and tokens may be the inner one.
    ``k_scale``, ``v_scale``: float32 [pages, heads, page tokens / block] of the
    same layers, contiguous but for the layers.  A sequence's pages are named by its row of a page table."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @classmethod
    def new(cls, pages, heads, page_tokens, dim, block=None, layers=None, device=None):
        """An empty cache (its memory is not set); ``block`` tokens share a scale, by default a page's."""
        lead = () if layers is None else (layers,)
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        shape, blocks = lead + (pages, heads), page_tokens // (page_tokens if block is None else block)
        entries = [torch.empty(*shape, page_tokens, dim, dtype=torch.float8_e4m3fn, device=device) for _ in range(2)]
        scales = [torch.empty(*shape, blocks, dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*entries, *scales)

    def layer(self, i):
        """The cache of one layer."""
        return PagedCache(*(t[i] for t in self))


def _strides_differ(a, b):
    """Of two tensors of one shape, those that are used."""
    return any(n > 1 and i != j for n, i, j in zip(a.shape, a.stride(), b.stride()))


def _cache(cache, dev, layered):
    """sv_cache of (k, v, k_scale, v_scale), checked."""
    k, v, ks, vs = cache
    f8, f32 = torch.float8_e4m3fn, torch.float32
    st, shape, ss, scales = k.stride(), k.shape, ks.stride(), ks.shape
    dim = len(shape)
    if dim != 4 and not (layered and dim == 5):
        raise ValueError(f"cache k: {dim} dimensions, expected {'4 or 5' if layered else 4}")
    if k.dtype != f8 or v.dtype != f8 or ks.dtype != f32 or vs.dtype != f32:
        raise TypeError(f"cache: dtypes {k.dtype}, {v.dtype}, {ks.dtype}, {vs.dtype}, expected {f8} twice and {f32} twice")
    if k.device != dev or v.device != dev or ks.device != dev or vs.device != dev:
        raise ValueError(f"cache: on {k.device}, {v.device}, {ks.device}, {vs.device}, expected {dev}")
    if v.shape != shape or (v.stride() != st and _strides_differ(v, k)):
        raise ValueError("cache v: shape and strides differ from those of k")
    if vs.shape != scales or (vs.stride() != ss and _strides_differ(vs, ks)):
        raise ValueError("cache v_scale: shape and strides differ from those of k_scale")
    pages, heads, tokens, d = shape[-4:]
    per = scales[-1]
    if scales[:-1] != shape[:-2] or per < 1 or tokens % per:
        raise ValueError(f"cache k_scale: shape {tuple(scales)} does not go with k {tuple(shape)}")
    if st[-1] != 1 and d > 1:
        raise ValueError("cache k: the entries of a token must be contiguous")
    if (per > 1 and ss[-1] != 1) or (heads > 1 and ss[-2] != per) or (pages > 1 and ss[-3] != heads * per):
        raise ValueError("cache k_scale must be contiguous")
    # a stride over one entry may be anything: it is not used
    layers = shape[0] if dim == 5 else 1
    return SvCache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), st[0] if layers > 1 else 0,
                   st[-4] if pages > 1 else 0, st[-3] if heads > 1 else 0, st[-2] if tokens > 1 else d,
                   ss[0] if layers > 1 else 0, layers, pages, heads, tokens, tokens // per, d)


def _step(dev, page_table, context, node_start):
    """Checks of a step's page table, contexts and node ranges; returns the table's pointer, stride and columns and B."""
    i32 = torch.int32
    stride = _check_rows(page_table, "page_table", 2, i32, dev)[0]
    B, cols = page_table.shape
    _check(context, "context", (B,), i32, dev)
    if node_start is not None:
        _check(node_start, "node_start", (B + 1,), i32, dev)
    return page_table.data_ptr(), stride, cols, B


def cache_write(cache, k, v, page_table, context, node_start, max_nodes=None, stream=None):
    """Write a step's (or a prompt's) keys and values into the pages of a ``PagedCache``, in 8 bits.

    ``k``, ``v`` [nodes + B, heads, dim] (bfloat16 or float32, entries contiguous):
    each sequence's root row, then its nodes' rows, as ``verify_tree`` takes them;
    they go to the positions ``context[b]``, ``context[b] + 1``, ...  ``page_table``
    [B, columns], ``context`` [B] and ``node_start`` [B + 1] are int32.  A prompt
    of n tokens is a sequence with n - 1 nodes.  ``max_nodes`` bounds a sequence's
    nodes (default: the number of nodes; blocks of threads are launched for as many
    in every sequence, so that a batch of prompts should name its longest: 32 prompts
    of up to 2048 tokens take 593 us without it, 54 with it).  How scales follow the entries:
    ``spec_verify_cache_write`` in include/spec_verify.h."""
    dev = _cuda_device(k, "k")
    c = _cache(cache, dev, False)
    table, t_stride, cols, B = _step(dev, page_table, context, node_start)
    ks = _check_rows(k, "k", 3, None, dev)
    vs = _check_rows(v, "v", 3, k.dtype, dev)
    rows = k.shape[0]
    if rows < B or k.shape[1:] != (c.heads, c.dim) or v.shape != k.shape:
        raise ValueError(f"k, v: shapes {tuple(k.shape)}, {tuple(v.shape)}, expected (nodes + {B}, {c.heads}, {c.dim})")
    if max_nodes is None:
        max_nodes = rows - B
    rc = spec_verify_cache_write(ctypes.byref(c), k.data_ptr(), v.data_ptr(), _dt(k), ks[0], ks[1], vs[0], vs[1], table,
                                 t_stride, cols, context.data_ptr(), node_start.data_ptr(), B, rows - B, max_nodes, dev.index,
                                 _stream(dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_cache_write")


def cache_keep(cache, path, accepted_len, page_table, context, out=None, stream=None):
    """Keep the cache's rows of the accepted drafts: ``path`` and ``accepted_len`` as ``verify_tree`` returns them.

    In every layer of the cache (``PagedCache``, with or without layers in front)
    the rows of a sequence's path move to the positions behind its root; what
    lies behind them is free.  Returns the new contexts (``out``, or a new
    tensor): ``context + 1 + accepted_len``; they are unchanged where nothing
    could be kept (``spec_verify_cache_keep`` in include/spec_verify.h)."""
    dev = _cuda_device(path, "path")
    c = _cache(cache, dev, True)
    table, t_stride, cols, B = _step(dev, page_table, context, None)
    i32 = torch.int32
    _check(path, "path", (B, path.shape[-1]), i32, dev)
    _check(accepted_len, "accepted_len", (B,), i32, dev)
    if out is None:
        out = _new(dev, stream, lambda: torch.empty(B, dtype=i32, device=dev))
    else:
        _check(out, "out", (B,), i32, dev)
    rc = spec_verify_cache_keep(ctypes.byref(c), path.data_ptr(), path.shape[1], accepted_len.data_ptr(), table, t_stride,
                                cols, context.data_ptr(), out.data_ptr(), B, dev.index, _stream(dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_cache_keep")
    return out


def attend_tree(q, cache, page_table, context, node_start, parent=None, scale=None, max_nodes=None, out=None, stream=None):
    """Attention of drafted rows over a ``PagedCache`` that holds their keys and values already (``cache_write``).

    ``q`` [nodes + B, query heads, dim] (bfloat16, entries contiguous, rows and
    heads on multiples of 16 bytes): each sequence's root row, then its nodes'
    rows, as ``verify_tree`` takes them.  A
    row sees the ``context[b]`` committed positions, the root and its path
    (``parent`` [nodes]; None: chains).  Plain decoding has a ``node_start`` of
    zeros.  ``scale``: of the logits, by default dim ** -0.5.  ``max_nodes``
    bounds a sequence's nodes (default: the number of nodes, as far as
    SV_MAX_NODES; short chains and small trees want theirs named: a bound that holds
    few columns takes a narrower kernel and less workspace, 167 us instead of 176
    for 64 chains of five).  Returns bfloat16 rows shaped as ``q`` (``out``, or a new
    tensor).  No gradient is recorded."""
    dev = _cuda_device(q, "q")
    bf16 = torch.bfloat16
    c = _cache(cache, dev, False)
    table, t_stride, cols, B = _step(dev, page_table, context, node_start)
    qs = _check_rows(q, "q", 3, bf16, dev)
    rows, q_heads, d = q.shape
    if d != c.dim or rows < B:
        raise ValueError(f"q: shape {tuple(q.shape)}, expected (nodes + {B}, query heads, {c.dim})")
    total = rows - B
    if parent is not None:
        _check(parent, "parent", (total,), torch.int32, dev)
    if max_nodes is None:
        max_nodes = min(total, SV_MAX_NODES)
    if out is not None:
        _check_rows(out, "out", 3, bf16, dev)
        if out.shape != q.shape:
            raise ValueError(f"out: shape {tuple(out.shape)} != {tuple(q.shape)}")
    size = spec_verify_attend_workspace(c.heads, q_heads, d, max_nodes, dev.index)
    new, work = _new(dev, stream, lambda: (torch.empty(q.shape, dtype=bf16, device=dev) if out is None else out,
                                           torch.empty(size, dtype=torch.uint8, device=dev)))
    os = new.stride()
    rc = spec_verify_attend(ctypes.byref(c), q.data_ptr(), qs[0], qs[1], new.data_ptr(), os[0], os[1], q_heads,
                            d ** -0.5 if scale is None else float(scale), table, t_stride, cols, context.data_ptr(),
                            node_start.data_ptr(), _ptr(parent), B, total, max_nodes, work.data_ptr(), size, dev.index,
                            _stream(dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_attend")
    return new


class SpecVerifier:
    """A verifier handle for batches up to ``max_B`` with ``k`` drafts over ``V`` tokens."""

    def __init__(self, max_B: int, k: int, V: int, device: int = 0):
        self.max_B, self.k, self.V = int(max_B), int(k), int(V)
        self.device = torch.device("cuda", device)
        self.handle = spec_verify_init(max_B, k, V, device)

    def close(self):
        if self.handle:
            spec_verify_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def mark_next(self, ev_before: torch.cuda.Event, ev_after: torch.cuda.Event):
        """Time the next call's stream pass with two torch CUDA events (enable_timing=True,
        already recorded once so that torch has created them)."""
        if not ev_before.cuda_event or not ev_after.cuda_event:
            raise ValueError("record both events once before passing them (torch creates them lazily)")
        rc = spec_verify_mark_next(self.handle, ev_before.cuda_event, ev_after.cuda_event)
        if rc != SV_OK:
            raise SpecVerifyError(rc, "spec_verify_mark_next")

    def set_filters(self, target=(0, 1.0, 0.0), draft=(0, 1.0, 0.0)):
        """Sampler filters (top_k, top_p, min_p) of the target rows and of the
        draft rows for later calls; (0, 1.0, 0.0) is off."""
        rc = spec_verify_set_filters(self.handle, int(target[0]), float(target[1]), float(target[2]),
                                     int(draft[0]), float(draft[1]), float(draft[2]))
        if rc != SV_OK:
            raise SpecVerifyError(rc, "spec_verify_set_filters")

    def set_gate_policy(self, schedule=None, min_cum: float = 0.0):
        """Per-step thresholds (a sequence of floats in [0, 1], the last one
        repeating; None for none) and the cumulative floor (0 = off) of the
        gated sequences of later calls.  Raises on a malformed policy, which
        then leaves the previous one in place."""
        arr, n = None, 0
        if schedule is not None:
            vals = [float(x) for x in schedule]
            n = len(vals)
            arr = (ctypes.c_float * max(n, 1))(*vals)
        rc = spec_verify_set_gate_policy(self.handle, arr, n, float(min_cum))
        if rc != SV_OK:
            raise SpecVerifyError(rc, "spec_verify_set_gate_policy")

    def outputs(self, B: int):
        dev = self.device
        return dict(
            accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
            tokens=torch.empty(B, self.k + 1, dtype=torch.int32, device=dev),
            accept_prob=torch.empty(B, self.k, dtype=torch.float32, device=dev),
            flags=torch.empty(B, self.k, dtype=torch.int8, device=dev),
        )

    def run(self, Lt, Ld, D, temperature, gate_mode=SV_PLAIN, threshold=0.5, gate_per_seq=None,
            threshold_per_seq=None, seed=0, seq_offset=0, u_accept=None, u_residual=None,
            counters=None, row_stats=False, out=None, stream=None):
        """Verify device tensors; returns a dict of device output tensors."""
        B = Lt.shape[0]
        k, V, dev = self.k, self.V, self.device
        _check(Lt, "target_logits", (B, k + 1, V), device=dev)
        _check(Ld, "draft_logits", (B, k, V), device=dev)
        _check(D, "draft_tokens", (B, k), torch.int32, dev)
        if gate_per_seq is not None:
            _check(gate_per_seq, "gate_mode_per_seq", (B,), torch.uint8, dev)
        if threshold_per_seq is not None:
            _check(threshold_per_seq, "threshold_per_seq", (B,), torch.float32, dev)
        if u_accept is not None:
            _check(u_accept, "u_accept", (B, k), torch.float32, dev)
        if u_residual is not None:
            _check(u_residual, "u_residual", (B,), torch.float32, dev)
        if counters is not None:
            _check(counters, "counters", (8,), torch.int64, dev)
        o = _new(dev, stream, lambda: self.outputs(B)) if out is None else out
        rs = _new(dev, stream, lambda: torch.empty(B, 2 * k + 1, 2, dtype=torch.float32, device=dev)) if row_stats else None
        st = torch.cuda.current_stream(dev).cuda_stream if stream is None else stream
        rc = spec_verify_run_ex(self.handle, Lt.data_ptr(), _dt(Lt), Ld.data_ptr(), _dt(Ld),
                                D.data_ptr(), B, float(temperature), int(gate_mode),
                                float(threshold), _ptr(gate_per_seq), _ptr(threshold_per_seq),
                                int(seed), int(seq_offset), _ptr(u_accept), _ptr(u_residual),
                                o["accepted_len"].data_ptr(), o["tokens"].data_ptr(),
                                o["accept_prob"].data_ptr(), _ptr(o.get("flags")),
                                _ptr(counters), _ptr(rs), st)
        if rc != SV_OK:
            raise SpecVerifyError(rc, "spec_verify_run_ex")
        if rs is not None:
            o["row_stats"] = rs
        return o

    def run_hidden(self, target_hidden, target_head, draft_hidden, draft_head, D, temperature, target_bias=None,
                   draft_bias=None, cap=None, logits_dtype=torch.bfloat16, penalties=None, **kw):
        """Verify from hidden states: the output heads' products, penalties on the logits, then ``run``.

        ``target_hidden`` [B, k+1, H] with ``target_head`` [V, H];
        ``draft_hidden`` [B, k, H'] with ``draft_head`` [V, H'], or [k, V, H']
        for a head per position (all bfloat16), and biases [V] (or [k, V]).
        ``cap`` bounds both sides' logits (cap * tanh(z / cap)).  ``penalties``: what
        ``penalize`` takes by these names -- history, history_len, prompt_len,
        repetition, frequency, presence, bias -- for the rows of both sides, row j
        of which stands behind D[:, :j]; mask and mask_row for the target's [B *
        (k+1)] rows, draft_mask and draft_mask_row for the draft's [B * k] (a side
        without a mask is not masked); other names are refused.  ``kw``
        goes to ``run``; the result also holds target_logits and draft_logits, as
        they were verified."""
        if penalties is not None:
            unknown = set(penalties) - RUN_HIDDEN_PENALTIES
            if unknown:
                raise TypeError(f"penalties: unknown names {sorted(unknown)}, expected some of {sorted(RUN_HIDDEN_PENALTIES)}")
        B, k, V, dev = target_hidden.shape[0], self.k, self.V, self.device
        _check(target_hidden, "target_hidden", (B, k + 1, target_hidden.shape[-1]), torch.bfloat16, dev)
        _check(draft_hidden, "draft_hidden", (B, k, draft_hidden.shape[-1]), torch.bfloat16, dev)
        stream = kw.get("stream")
        Lt, Ld = _new(dev, stream, lambda: [torch.empty(B, n, V, dtype=logits_dtype, device=dev) for n in (k + 1, k)])
        act = dict(activation="none" if cap is None else "softcap", cap=cap or 0.0, stream=stream)
        linear(target_hidden.view(B * (k + 1), target_hidden.shape[-1]), target_head, bias=target_bias,
               out=Lt.view(B * (k + 1), V), **act)
        if draft_head.dim() == 3:
            linear(draft_hidden.transpose(0, 1), draft_head, bias=draft_bias, out=Ld.transpose(0, 1), **act)
        else:
            linear(draft_hidden.view(B * k, draft_hidden.shape[-1]), draft_head, bias=draft_bias,
                   out=Ld.view(B * k, V), **act)
        if penalties is not None:
            _check(D, "draft_tokens", (B, k), torch.int32, dev)
            both = {name: t for name, t in penalties.items() if "mask" not in name}
            tokens, start = _new(dev, stream, lambda: (D[:, :k - 1].reshape(-1), [
                torch.arange(B + 1, dtype=torch.int32, device=dev) * n for n in (k, k - 1)]))
            penalize(Lt.view(B * (k + 1), V), tokens=D.view(-1), parent=None, node_start=start[0], max_nodes=k,
                     mask=penalties.get("mask"), mask_row=penalties.get("mask_row"), out=Lt.view(B * (k + 1), V),
                     stream=stream, **both)
            penalize(Ld.view(B * k, V), tokens=tokens, parent=None, node_start=start[1], max_nodes=k - 1,
                     mask=penalties.get("draft_mask"), mask_row=penalties.get("draft_mask_row"), out=Ld.view(B * k, V),
                     stream=stream, **both)
        out = self.run(Lt, Ld, D, temperature, **kw)
        out["target_logits"], out["draft_logits"] = Lt, Ld
        return out

    def diagnostics(self, Lt, Ld, D, temperature, gate_mode=SV_PLAIN, threshold=0.5,
                    gate_per_seq=None, threshold_per_seq=None, out=None, stream=None):
        """Closed-form acceptance of every draft position: a dict of [B, k]
        float device tensors min_sum (sum min(p, mu)), pq_sum (sum p q) and
        argmax_q (q at the first largest p); NaN where the rows are invalid."""
        B = Lt.shape[0]
        k, V, dev = self.k, self.V, self.device
        _check(Lt, "target_logits", (B, k + 1, V), device=dev)
        _check(Ld, "draft_logits", (B, k, V), device=dev)
        _check(D, "draft_tokens", (B, k), torch.int32, dev)
        if gate_per_seq is not None:
            _check(gate_per_seq, "gate_mode_per_seq", (B,), torch.uint8, dev)
        if threshold_per_seq is not None:
            _check(threshold_per_seq, "threshold_per_seq", (B,), torch.float32, dev)
        if out is None:
            out = _new(dev, stream, lambda: {key: torch.empty(B, k, dtype=torch.float32, device=dev)
                                             for key in ("min_sum", "pq_sum", "argmax_q")})
        st = torch.cuda.current_stream(dev).cuda_stream if stream is None else stream
        rc = spec_verify_diagnostics(self.handle, Lt.data_ptr(), _dt(Lt), Ld.data_ptr(), _dt(Ld),
                                     D.data_ptr(), B, float(temperature), int(gate_mode),
                                     float(threshold), _ptr(gate_per_seq), _ptr(threshold_per_seq),
                                     _ptr(out.get("min_sum")), _ptr(out.get("pq_sum")),
                                     _ptr(out.get("argmax_q")), st)
        if rc != SV_OK:
            raise SpecVerifyError(rc, "spec_verify_diagnostics")
        return out

    def run_host(self, Lt, Ld, D, temperature, gate_mode=SV_PLAIN, threshold=0.5,
                 gate_per_seq=None, threshold_per_seq=None, seed=0, out=None, counters=None,
                 stream=None):
        """Verify host (ideally pinned) tensors through the host-buffer entry point."""
        B = Lt.shape[0]
        k, V, cpu = self.k, self.V, torch.device("cpu")
        _check(Lt, "target_logits", (B, k + 1, V), device=cpu)
        _check(Ld, "draft_logits", (B, k, V), device=cpu)
        _check(D, "draft_tokens", (B, k), torch.int32, cpu)
        if out is None:
            out = dict(accepted_len=torch.empty(B, dtype=torch.int32),
                       tokens=torch.empty(B, k + 1, dtype=torch.int32),
                       accept_prob=torch.empty(B, k, dtype=torch.float32),
                       flags=torch.empty(B, k, dtype=torch.int8))
        st = torch.cuda.current_stream(self.device).cuda_stream if stream is None else stream
        rc = spec_verify_run_host(self.handle, Lt.data_ptr(), _dt(Lt), Ld.data_ptr(), _dt(Ld),
                                  D.data_ptr(), B, float(temperature), int(gate_mode),
                                  float(threshold), _ptr(gate_per_seq), _ptr(threshold_per_seq),
                                  int(seed), out["accepted_len"].data_ptr(),
                                  out["tokens"].data_ptr(), out["accept_prob"].data_ptr(),
                                  _ptr(out.get("flags")), _ptr(counters), st)
        if rc != SV_OK:
            raise SpecVerifyError(rc, "spec_verify_run_host")
        return out


def run_noalloc(Lt, Ld, D, temperature, gate_mode=SV_PLAIN, threshold=0.5, gate_per_seq=None,
                threshold_per_seq=None, seed=0, out=None, counters=None, stream=None):
    """Verify device tensors through the allocation-free entry point on their device.

    The outputs are the caller's tensors (``out``, or new ones made here by
    torch); the library itself allocates nothing.  Calls on one device must
    not overlap."""
    B, k1, V = Lt.shape
    k = k1 - 1
    dev = Lt.device
    _check(Lt, "target_logits", (B, k + 1, V), device=dev)
    _check(Ld, "draft_logits", (B, k, V), device=dev)
    _check(D, "draft_tokens", (B, k), torch.int32, dev)
    if out is None:
        out = _new(dev, stream, lambda: dict(
            accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
            tokens=torch.empty(B, k + 1, dtype=torch.int32, device=dev),
            accept_prob=torch.empty(B, k, dtype=torch.float32, device=dev),
            flags=torch.empty(B, k, dtype=torch.int8, device=dev)))
    with torch.cuda.device(dev):
        st = torch.cuda.current_stream(dev).cuda_stream if stream is None else stream
        rc = spec_verify_run_noalloc(Lt.data_ptr(), _dt(Lt), Ld.data_ptr(), _dt(Ld), D.data_ptr(), B,
                                     k, V, float(temperature), int(gate_mode), float(threshold),
                                     _ptr(gate_per_seq), _ptr(threshold_per_seq), int(seed),
                                     out["accepted_len"].data_ptr(), out["tokens"].data_ptr(),
                                     out["accept_prob"].data_ptr(), _ptr(out.get("flags")),
                                     _ptr(counters), st)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_run_noalloc")
    return out
