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
                   draft_bias=None, cap=None, logits_dtype=torch.bfloat16, **kw):
        """Verify from hidden states: the output heads' products, then ``run``.

        ``target_hidden`` [B, k+1, H] with ``target_head`` [V, H];
        ``draft_hidden`` [B, k, H'] with ``draft_head`` [V, H'], or [k, V, H']
        for a head per position (all bfloat16), and biases [V] (or [k, V]).
        ``cap`` bounds both sides' logits (cap * tanh(z / cap)).  ``kw`` goes to
        ``run``; the result also holds target_logits and draft_logits."""
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
