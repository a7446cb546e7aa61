"""What the operators around a verifying call refuse, on the host and before any launch: no GPU is needed, and no
call here could start one (every raw call has an argument that the entry point rejects first)."""
from __future__ import annotations

import pytest
import torch

import speculative_decoding_verification_online_gb300 as sv
from speculative_decoding_verification_online_gb300 import spec_verify as m


@pytest.fixture(scope="module", autouse=True)
def library():
    from speculative_decoding_verification_online_gb300 import build as B
    return B.build()


A = 1 << 20  # a multiple of every alignment, never read

LINEAR = dict(x=A, x_row=64, x_group=0, w=A, w_row=64, w_group=0, bias=None, bias_dt=0, bias_group=0, residual=None,
              residual_dt=0, residual_row=0, residual_group=0, y=A, y_dt=1, y_row=32, y_group=128, groups=2, M=4, N=32,
              K=64, act=0, cap=0.0, device=0, stream=None)
SOFTMAX = dict(logits=A, dt=1, logits_stride=10, rows=2, V=10, temperature=1.0, temperature_per_row=None, probs=A,
               probs_stride=10, device=0, stream=None)
TREE = dict(p=A, p_stride=10, q=A, q_stride=10, draft_rows=2, node_start=A, tokens=A, parent=A, draft_row=A, u_accept=A,
            u_pick=A, B=2, total_nodes=3, max_nodes=2, max_depth=2, V=10, siblings=0, accepted_len=A, out_tokens=A,
            path=A, accept_prob=A, flags=A, counters=A, device=0, stream=None)


def _call(fn, base, change):
    return fn(*dict(base, **change).values())


@pytest.mark.parametrize("change,status", [
    (dict(groups=-1), m.SV_EINVAL), (dict(M=-1), m.SV_EINVAL), (dict(N=-5), m.SV_EINVAL), (dict(K=-1), m.SV_EINVAL),
    (dict(y_dt=2), m.SV_EINVAL), (dict(bias=A, bias_dt=7), m.SV_EINVAL), (dict(residual=A, residual_dt=-1), m.SV_EINVAL),
    (dict(act=6), m.SV_EINVAL), (dict(act=-1), m.SV_EINVAL), (dict(act=5, cap=0.0), m.SV_EINVAL),
    (dict(act=5, cap=float("nan")), m.SV_EINVAL), (dict(act=5, cap=float("inf")), m.SV_EINVAL),
    (dict(x_row=-1), m.SV_EINVAL), (dict(y_group=-8), m.SV_EINVAL), (dict(w_row=1 << 40), m.SV_EUNSUPPORTED),
    (dict(x=None), m.SV_EINVAL), (dict(w=None), m.SV_EINVAL), (dict(y=None), m.SV_EINVAL), (dict(x=A + 1), m.SV_EINVAL),
    (dict(w=A + 1), m.SV_EINVAL), (dict(y=A + 1), m.SV_EINVAL), (dict(y_dt=0, y=A + 2), m.SV_EINVAL),
    (dict(bias=A + 1, bias_dt=1), m.SV_EINVAL), (dict(residual=A + 2, residual_dt=0), m.SV_EINVAL),
    (dict(y_row=31), m.SV_EINVAL), (dict(y_group=96), m.SV_EINVAL), (dict(y_row=64, y_group=33), m.SV_EINVAL),
    (dict(y_row=0), m.SV_EINVAL), (dict(y_group=0), m.SV_EINVAL),
    (dict(K=(1 << 30) + 1), m.SV_EUNSUPPORTED), (dict(N=(1 << 31) - 1, y_row=1 << 33, y_group=1 << 31), m.SV_EUNSUPPORTED),
])
def test_linear_refuses(change, status):
    assert _call(sv.spec_verify_linear, LINEAR, change) == status


@pytest.mark.parametrize("change", [dict(groups=0), dict(M=0), dict(N=0), dict(M=0, x=None, y=None)])
def test_linear_of_nothing_is_a_no_op(change):
    assert _call(sv.spec_verify_linear, LINEAR, change) == m.SV_OK


@pytest.mark.parametrize("change,status", [
    (dict(dt=3), m.SV_EINVAL), (dict(rows=-1), m.SV_EINVAL), (dict(V=0), m.SV_EINVAL),
    (dict(V=(1 << 22) + 1, probs_stride=1 << 23), m.SV_EUNSUPPORTED), (dict(temperature=-0.5), m.SV_EINVAL),
    (dict(temperature=float("nan")), m.SV_EINVAL), (dict(temperature=float("inf")), m.SV_EINVAL),
    (dict(logits=None), m.SV_EINVAL), (dict(probs=None), m.SV_EINVAL), (dict(logits=A + 1), m.SV_EINVAL),
    (dict(dt=0, logits=A + 2), m.SV_EINVAL), (dict(probs=A + 2), m.SV_EINVAL),
    (dict(temperature_per_row=A + 1), m.SV_EINVAL), (dict(probs_stride=9), m.SV_EINVAL),
    (dict(logits_stride=-10), m.SV_EINVAL),
])
def test_softmax_refuses(change, status):
    assert _call(sv.spec_verify_softmax, SOFTMAX, change) == status


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), m.SV_EINVAL), (dict(total_nodes=-1), m.SV_EINVAL), (dict(max_nodes=-1), m.SV_EINVAL),
    (dict(max_depth=-1), m.SV_EINVAL), (dict(draft_rows=-1), m.SV_EINVAL), (dict(V=0), m.SV_EINVAL),
    (dict(siblings=2), m.SV_EINVAL), (dict(V=(1 << 22) + 1), m.SV_EUNSUPPORTED), (dict(max_nodes=257), m.SV_EUNSUPPORTED),
    (dict(max_depth=3), m.SV_EINVAL), (dict(p=None), m.SV_EINVAL), (dict(q=None), m.SV_EINVAL),
    (dict(node_start=None), m.SV_EINVAL), (dict(tokens=None), m.SV_EINVAL), (dict(parent=None), m.SV_EINVAL),
    (dict(draft_row=None), m.SV_EINVAL), (dict(u_accept=None), m.SV_EINVAL), (dict(u_pick=None), m.SV_EINVAL),
    (dict(accepted_len=None), m.SV_EINVAL), (dict(out_tokens=None), m.SV_EINVAL), (dict(p_stride=-1), m.SV_EINVAL),
    (dict(q_stride=-1), m.SV_EINVAL), (dict(p=A + 2), m.SV_EINVAL), (dict(q=A + 1), m.SV_EINVAL),
    (dict(u_pick=A + 1), m.SV_EINVAL), (dict(counters=A + 4), m.SV_EINVAL), (dict(path=A + 2), m.SV_EINVAL),
])
def test_tree_refuses(change, status):
    assert _call(sv.spec_verify_tree, TREE, change) == status


def test_batches_of_nothing_are_no_ops():
    assert _call(sv.spec_verify_tree, TREE, dict(B=0, p=None, u_pick=None)) == m.SV_OK
    assert _call(sv.spec_verify_softmax, SOFTMAX, dict(rows=0, logits=None, probs=None)) == m.SV_OK


def test_python_calls_refuse_tensors_that_are_not_on_a_gpu():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sv.linear(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        sv.softmax(x, 1.0)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sv.verify_tree(x.float(), None, i, i, i, i, i.float(), i.float())


class _OnGpu:
    """Stands for a CUDA tensor of which only shape, type and place are looked at."""

    def __init__(self, shape, dtype=torch.bfloat16, strides=None, device="cuda:0"):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self.strides = strides or torch.empty(shape, device="meta").stride()

    def stride(self):
        return self.strides

    def data_ptr(self):
        return A

    def is_contiguous(self):
        return True


def test_python_linear_refuses_shapes_types_and_places():
    x, w = _OnGpu((4, 8)), _OnGpu((16, 8))
    for args, kw, error in (
            ((x, _OnGpu((8,))), {}, ValueError), ((x, _OnGpu((16, 8), torch.float32)), {}, TypeError),
            ((_OnGpu((4, 8), torch.float16), w), {}, TypeError), ((_OnGpu((4, 9)), w), {}, ValueError),
            ((_OnGpu((2, 4, 8)), w), {}, ValueError), ((_OnGpu((3, 4, 8)), _OnGpu((2, 16, 8))), {}, ValueError),
            ((_OnGpu((4, 8), strides=(1, 4)), w), {}, ValueError), ((x, _OnGpu((16, 8), device="cuda:1")), {}, ValueError),
            ((x, w), dict(activation="tanh", out=_OnGpu((4, 16))), ValueError),
            ((x, w), dict(out=_OnGpu((4, 15))), ValueError),
            ((x, w), dict(out=_OnGpu((4, 16), torch.float32), out_dtype=torch.bfloat16), TypeError),
            ((x, w), dict(out=_OnGpu((4, 16)), bias=_OnGpu((4, 16))), ValueError),
            ((x, w), dict(out=_OnGpu((4, 16)), bias=_OnGpu((17,))), ValueError),
            ((x, w), dict(out=_OnGpu((4, 16)), residual=_OnGpu((16, 4))), ValueError)):
        with pytest.raises(error):
            sv.linear(*args, **kw)


def test_python_softmax_and_tree_refuse_shapes_and_types():
    x = _OnGpu((4, 8), torch.float32)
    with pytest.raises(ValueError):
        sv.softmax(_OnGpu((8,), torch.float32), 1.0)
    with pytest.raises(ValueError):
        sv.softmax(x, 1.0, out=_OnGpu((4, 9), torch.float32))
    with pytest.raises(TypeError):
        sv.softmax(x, 1.0, out=_OnGpu((4, 8)))
    i32, f32 = torch.int32, torch.float32
    good = dict(target_probs=_OnGpu((5, 8), f32), draft_probs=_OnGpu((2, 8), f32), tokens=_OnGpu((3,), i32),
                parent=_OnGpu((3,), i32), draft_row=_OnGpu((5,), i32), node_start=_OnGpu((3,), i32),
                u_accept=_OnGpu((3,), f32), u_pick=_OnGpu((2,), f32))
    for name, t, error in (("target_probs", _OnGpu((4, 8), f32), ValueError), ("target_probs", _OnGpu((5, 8)), TypeError),
                           ("draft_probs", _OnGpu((2, 7), f32), ValueError), ("tokens", _OnGpu((3,), torch.int64), TypeError),
                           ("parent", _OnGpu((2,), i32), ValueError), ("draft_row", _OnGpu((3,), i32), ValueError),
                           ("node_start", _OnGpu((2,), i32), ValueError), ("u_accept", _OnGpu((3,), torch.float64), TypeError),
                           ("u_pick", _OnGpu((3,), f32), ValueError),
                           ("draft_row", _OnGpu((5,), i32, device="cuda:1"), ValueError)):
        with pytest.raises(error):
            sv.verify_tree(**dict(good, **{name: t}))


@pytest.mark.parametrize("cap", [1e-45, 1e-40, 2.0 ** -128])
def test_linear_refuses_caps_without_a_finite_reciprocal(cap):
    # no call of a cap that is taken: its groups are 0
    assert _call(sv.spec_verify_linear, LINEAR, dict(act=5, cap=cap)) == m.SV_EINVAL
    assert _call(sv.spec_verify_linear, LINEAR, dict(act=5, cap=cap, groups=0)) == m.SV_EINVAL
    assert _call(sv.spec_verify_linear, LINEAR, dict(act=5, cap=2.0 ** -127, groups=0)) == m.SV_OK
