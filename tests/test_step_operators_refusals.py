"""What the operators around a tree's target pass refuse, on the host and before any launch: no GPU is needed, and no call
here could start one (every raw call has an argument that the entry point rejects first)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import speculative_decoding_verification_online_gb300 as sv
from speculative_decoding_verification_online_gb300 import spec_verify as m
from tests.test_operators_refusals import A, _call, _OnGpu


@pytest.fixture(scope="module", autouse=True)
def library():
    from speculative_decoding_verification_online_gb300 import build as B
    return B.build()


FAR = 1 << 30  # nowhere near A

PENALTIES = dict(logits=A, dt=1, logits_stride=10, out=A + FAR, out_dt=1, out_stride=10, V=10, history=A, history_stride=4,
                 history_cap=4, history_len=A, prompt_len=A, node_tokens=A, parent=A, node_start=A, B=2, total_nodes=3,
                 max_nodes=2, repetition=A, frequency=A, presence=A, bias_start=A, bias_tokens=A, bias_values=A,
                 total_biases=4, mask=A, mask_stride=1, mask_rows=5, mask_row=A, device=0, stream=None)
CACHE = dict(k=A, v=A, k_scale=A, v_scale=A, layer_stride=0, page_stride=4096, head_stride=1024, token_stride=64,
             scale_layer_stride=0, layers=1, pages=9, heads=4, page_tokens=16, block=8, dim=64)
WRITE = dict(cache=None, k=A, v=A, dt=1, k_row=256, k_head=64, v_row=256, v_head=64, page_table=A, table_stride=3,
             table_cols=3, context=A, node_start=A, B=2, total_nodes=3, max_nodes=3, device=0, stream=None)
KEEP = dict(cache=None, path=A, max_depth=2, accepted_len=A, page_table=A, table_stride=3, table_cols=3, context=A,
            new_context=A + 64, B=2, device=0, stream=None)
ATTEND = dict(cache=None, q=A, q_row=512, q_head=64, out=A + FAR, out_row=512, out_head=64, q_heads=8, scale=0.1,
              page_table=A, table_stride=3, table_cols=3, context=A, node_start=A, parent=A, B=2, total_nodes=3, max_nodes=3,
              workspace=A, workspace_bytes=1 << 40, device=0, stream=None)


def _cached(fn, base, change, cache=None):
    c = sv.SvCache(**dict(CACHE, **(cache or {})))
    return _call(fn, base, dict(dict(cache=ctypes.byref(c)), **change))


@pytest.mark.parametrize("change,status", [
    (dict(dt=2), m.SV_EINVAL), (dict(out_dt=-1), m.SV_EINVAL), (dict(V=0), m.SV_EINVAL), (dict(B=-1), m.SV_EINVAL),
    (dict(total_nodes=-1), m.SV_EINVAL), (dict(max_nodes=-1), m.SV_EINVAL), (dict(history_cap=-1), m.SV_EINVAL),
    (dict(total_biases=-1), m.SV_EINVAL), (dict(mask_rows=-1), m.SV_EINVAL), (dict(V=(1 << 22) + 1), m.SV_EUNSUPPORTED),
    (dict(max_nodes=257), m.SV_EUNSUPPORTED), (dict(history_cap=1 << 30), m.SV_EUNSUPPORTED),
    (dict(total_nodes=2 ** 31 - 1), m.SV_EUNSUPPORTED), (dict(logits=None), m.SV_EINVAL), (dict(out=None), m.SV_EINVAL),
    (dict(history=None), m.SV_EINVAL), (dict(history_len=None), m.SV_EINVAL), (dict(node_start=None), m.SV_EINVAL),
    (dict(node_tokens=None), m.SV_EINVAL), (dict(bias_tokens=None), m.SV_EINVAL), (dict(bias_values=None), m.SV_EINVAL),
    (dict(logits=A + 1), m.SV_EINVAL), (dict(out_dt=0, out=A + FAR + 2), m.SV_EINVAL), (dict(mask=A + 2), m.SV_EINVAL),
    (dict(frequency=A + 1), m.SV_EINVAL), (dict(out_stride=9), m.SV_EINVAL), (dict(logits_stride=-1), m.SV_EINVAL),
    (dict(history_stride=-4), m.SV_EINVAL), (dict(V=40, logits_stride=40, out_stride=40), m.SV_EINVAL),
    (dict(mask_row=None, mask_rows=4), m.SV_EINVAL), (dict(out=A, out_stride=12), m.SV_EINVAL),
    (dict(out=A, out_dt=0), m.SV_EINVAL), (dict(out=A + 4), m.SV_EINVAL)])
def test_penalties_refuse(change, status):
    assert _call(sv.spec_verify_penalties, PENALTIES, change) == status


CACHES = [(None, m.SV_EINVAL)] + [(c, m.SV_EINVAL) for c in (
    dict(layers=0), dict(pages=-1), dict(heads=0), dict(page_tokens=24), dict(block=3), dict(block=32), dict(token_stride=48),
    dict(page_stride=4097), dict(head_stride=-16), dict(k=None), dict(v_scale=None), dict(k=A + 8), dict(k_scale=A + 2))] + [
    (c, m.SV_EUNSUPPORTED) for c in (dict(page_tokens=8), dict(page_tokens=512), dict(dim=96), dict(dim=256, token_stride=256),
                                     dict(page_stride=1 << 40))]


@pytest.mark.parametrize("fn,base", [(m.spec_verify_cache_write, WRITE), (m.spec_verify_cache_keep, KEEP),
                                     (m.spec_verify_attend, ATTEND)])
@pytest.mark.parametrize("cache,status", CACHES)
def test_caches_that_are_refused(fn, base, cache, status):
    if cache is None:
        assert _call(fn, base, {}) == status
    else:
        assert _cached(fn, base, {}, cache) == status


@pytest.mark.parametrize("change,status", [
    (dict(dt=5), m.SV_EINVAL), (dict(k=None), m.SV_EINVAL), (dict(v=None), m.SV_EINVAL), (dict(context=None), m.SV_EINVAL),
    (dict(node_start=None), m.SV_EINVAL), (dict(page_table=None), m.SV_EINVAL), (dict(table_cols=-1), m.SV_EINVAL),
    (dict(table_stride=-1), m.SV_EINVAL), (dict(B=-2), m.SV_EINVAL), (dict(total_nodes=-1), m.SV_EINVAL),
    (dict(max_nodes=-1), m.SV_EINVAL), (dict(k_row=-1), m.SV_EINVAL), (dict(v_head=1 << 40), m.SV_EUNSUPPORTED),
    (dict(k=A + 1), m.SV_EINVAL), (dict(context=A + 1), m.SV_EINVAL), (dict(total_nodes=2 ** 31 - 2), m.SV_EUNSUPPORTED),
    (dict(B=1 << 28, max_nodes=1 << 20, total_nodes=1 << 20), m.SV_EUNSUPPORTED)])
def test_cache_write_refuses(change, status):
    assert _cached(sv.spec_verify_cache_write, WRITE, change) == status


def test_calls_that_work_on_one_layer_refuse_more():
    two = dict(layers=2, layer_stride=1 << 20, scale_layer_stride=1 << 10)
    assert _cached(sv.spec_verify_cache_write, WRITE, {}, two) == m.SV_EINVAL
    assert _cached(sv.spec_verify_attend, ATTEND, {}, two) == m.SV_EINVAL


@pytest.mark.parametrize("change,status", [
    (dict(path=None), m.SV_EINVAL), (dict(accepted_len=None), m.SV_EINVAL), (dict(context=None), m.SV_EINVAL),
    (dict(new_context=A), m.SV_EINVAL), (dict(max_depth=-1), m.SV_EINVAL), (dict(max_depth=257), m.SV_EUNSUPPORTED),
    (dict(B=-1), m.SV_EINVAL), (dict(new_context=A + 66), m.SV_EINVAL), (dict(page_table=A + 2), m.SV_EINVAL),
    (dict(B=2 ** 31 - 1), m.SV_EUNSUPPORTED)])
def test_cache_keep_refuses(change, status):
    assert _cached(sv.spec_verify_cache_keep, KEEP, change) == status


@pytest.mark.parametrize("change,status", [
    (dict(q_heads=0), m.SV_EINVAL), (dict(q_heads=6), m.SV_EINVAL), (dict(scale=float("nan")), m.SV_EINVAL),
    (dict(scale=float("inf")), m.SV_EINVAL), (dict(max_nodes=257), m.SV_EUNSUPPORTED), (dict(q=None), m.SV_EINVAL),
    (dict(out=None), m.SV_EINVAL), (dict(q=A + 2), m.SV_EINVAL), (dict(q_row=508), m.SV_EINVAL), (dict(q_head=-64), m.SV_EINVAL),
    (dict(out=A + FAR + 1), m.SV_EINVAL), (dict(out=A), m.SV_EINVAL), (dict(out_head=32), m.SV_EINVAL),
    (dict(out_row=64), m.SV_EINVAL), (dict(context=None), m.SV_EINVAL), (dict(parent=A + 1), m.SV_EINVAL),
    (dict(workspace=A + 8), m.SV_EINVAL), (dict(q_row=1 << 40), m.SV_EUNSUPPORTED), (dict(B=-1), m.SV_EINVAL)])
def test_attend_refuses(change, status):
    assert _cached(sv.spec_verify_attend, ATTEND, change) == status


@pytest.mark.parametrize("change", [
    dict(new_context=A + 4), dict(context=A + FAR, new_context=A), dict(context=A + FAR, new_context=A + 4),
    dict(context=A + FAR, accepted_len=A + FAR, new_context=A + 12),
    dict(context=A + FAR, accepted_len=A + FAR, new_context=A - 4)])
def test_cache_keep_refuses_new_contexts_over_what_it_reads(change):
    assert _cached(sv.spec_verify_cache_keep, KEEP, change) == m.SV_EINVAL


@pytest.mark.parametrize("scale", [1.01 * 2.0 ** 126, -3e38])
def test_attend_refuses_scales_that_leave_fp32(scale):
    assert _cached(sv.spec_verify_attend, ATTEND, dict(scale=scale)) == m.SV_EUNSUPPORTED


def test_batches_of_nothing_are_no_ops():
    assert _call(sv.spec_verify_penalties, PENALTIES, dict(B=0, logits=None, out=None)) == m.SV_OK
    assert _cached(sv.spec_verify_cache_write, WRITE, dict(B=0, k=None)) == m.SV_OK
    assert _cached(sv.spec_verify_cache_keep, KEEP, dict(B=0, path=None)) == m.SV_OK
    assert _cached(sv.spec_verify_attend, ATTEND, dict(B=0, q=None, out=None)) == m.SV_OK


def test_python_calls_refuse_tensors_that_are_not_on_a_gpu():
    x, i = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    c = [torch.zeros(1, 4, 16, 64).to(torch.float8_e4m3fn)] * 2 + [torch.zeros(1, 4, 1)] * 2
    for call in (lambda: sv.penalize(x, i.view(1, 2), i, i, i, i), lambda: sv.cache_write(c, q, q, i.view(1, 2), i, i),
                 lambda: sv.cache_keep(c, i.view(1, 2), i, i.view(1, 2), i), lambda: sv.attend_tree(q, c, i.view(1, 2), i, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


I32, F32, BF16, F8 = torch.int32, torch.float32, torch.bfloat16, torch.float8_e4m3fn


def test_python_penalize_refuses_shapes_and_types():
    good = dict(logits=_OnGpu((5, 40)), history=_OnGpu((2, 7), I32), history_len=_OnGpu((2,), I32), tokens=_OnGpu((3,), I32),
                parent=_OnGpu((3,), I32), node_start=_OnGpu((3,), I32), prompt_len=_OnGpu((2,), I32),
                repetition=_OnGpu((2,), F32), bias=(_OnGpu((3,), I32), _OnGpu((6,), I32), _OnGpu((6,), F32)),
                mask=_OnGpu((5, 2), I32))
    for name, t, error in (
            ("logits", _OnGpu((4, 40)), ValueError), ("logits", _OnGpu((5, 40), strides=(1, 5)), ValueError),
            ("history", _OnGpu((3, 7), I32), ValueError), ("history", _OnGpu((2, 7), torch.int64), TypeError),
            ("history_len", _OnGpu((2,), torch.int64), TypeError), ("parent", _OnGpu((4,), I32), ValueError),
            ("node_start", _OnGpu((2,), I32), ValueError), ("prompt_len", _OnGpu((3,), I32), ValueError),
            ("repetition", _OnGpu((2,)), TypeError), ("mask", _OnGpu((5, 1), I32), ValueError),
            ("mask", _OnGpu((4, 2), I32), ValueError), ("mask", None, ValueError),
            ("bias", (_OnGpu((2,), I32), _OnGpu((6,), I32), _OnGpu((6,), F32)), ValueError),
            ("bias", (_OnGpu((3,), I32), _OnGpu((6,), I32), _OnGpu((5,), F32)), ValueError),
            ("out", _OnGpu((5, 41)), ValueError), ("out", _OnGpu((5, 40), torch.float16), TypeError),
            ("tokens", _OnGpu((3,), I32, device="cuda:1"), ValueError)):
        kw = dict(good, **{name: t})
        if name == "mask" and t is None:
            kw["mask_row"] = _OnGpu((5,), I32)
        with pytest.raises(error):
            sv.penalize(**dict(dict(out=_OnGpu((5, 40))), **kw))


def _cache(**change):
    c = dict(k=_OnGpu((9, 4, 16, 64), F8), v=_OnGpu((9, 4, 16, 64), F8), k_scale=_OnGpu((9, 4, 2), F32),
             v_scale=_OnGpu((9, 4, 2), F32))
    c.update(change)
    return sv.PagedCache(**c)


BAD_CACHES = [
    (dict(k=_OnGpu((9, 4, 16, 64))), TypeError), (dict(v=_OnGpu((9, 4, 16, 32), F8)), ValueError),
    (dict(v=_OnGpu((9, 4, 16, 64), F8, (4096, 64, 256, 1))), ValueError), (dict(k_scale=_OnGpu((9, 4, 3), F32)), ValueError),
    (dict(k_scale=_OnGpu((9, 5, 2), F32), v_scale=_OnGpu((9, 5, 2), F32)), ValueError),
    (dict(v_scale=_OnGpu((9, 4, 2))), TypeError), (dict(k_scale=_OnGpu((9, 4, 2), F32, (2, 18, 1))), ValueError),
    (dict(k=_OnGpu((9, 4, 16, 64), F8, device="cuda:1")), ValueError),
    (dict(k_scale=_OnGpu((9, 4, 2), F32, (10, 2, 1)), v_scale=_OnGpu((9, 4, 2), F32, (10, 2, 1))), ValueError)]


@pytest.mark.parametrize("change,error", BAD_CACHES)
def test_python_calls_refuse_caches(change, error):
    table, two, three = _OnGpu((2, 3), I32), _OnGpu((2,), I32), _OnGpu((3,), I32)
    q = _OnGpu((5, 4, 64))
    c = _cache(**change)
    for call in (lambda: sv.cache_write(c, q, q, table, two, three), lambda: sv.cache_keep(c, _OnGpu((2, 3), I32), two, table, two),
                 lambda: sv.attend_tree(q, c, table, two, three, out=q)):
        with pytest.raises(error):
            call()


def test_python_cache_calls_refuse_shapes_and_types():
    c, table, two, three, q = _cache(), _OnGpu((2, 3), I32), _OnGpu((2,), I32), _OnGpu((3,), I32), _OnGpu((5, 4, 64))
    for args, error in (
            ((c, _OnGpu((5, 3, 64)), _OnGpu((5, 3, 64)), table, two, three), ValueError),
            ((c, q, _OnGpu((5, 4, 64), F32), table, two, three), TypeError), ((c, q, _OnGpu((4, 4, 64)), table, two, three), ValueError),
            ((c, _OnGpu((1, 4, 64)), _OnGpu((1, 4, 64)), table, two, three), ValueError),
            ((c, q, q, _OnGpu((2, 3), torch.int64), two, three), TypeError), ((c, q, q, table, three, three), ValueError),
            ((c, q, q, table, two, two), ValueError), ((c, _OnGpu((5, 4, 64), torch.float16), _OnGpu((5, 4, 64), torch.float16), table, two, three), TypeError)):
        with pytest.raises(error):
            sv.cache_write(*args)
    path = _OnGpu((2, 4), I32)
    for args, error in (((c, _OnGpu((3, 4), I32), two, table, two), ValueError), ((c, path, three, table, two), ValueError),
                        ((c, path, two, table, _OnGpu((2,), torch.int64)), TypeError)):
        with pytest.raises(error):
            sv.cache_keep(*args, out=two)
    for args, kw, error in (
            ((_OnGpu((5, 4, 128)), c, table, two, three), {}, ValueError), ((_OnGpu((5, 4, 64), F32), c, table, two, three), {}, TypeError),
            ((q, c, table, two, three, _OnGpu((4,), I32)), {}, ValueError), ((q, c, table, two, three), dict(out=_OnGpu((5, 4, 64), F32)), TypeError),
            ((q, c, table, two, three), dict(out=_OnGpu((5, 3, 64))), ValueError)):
        with pytest.raises(error):
            sv.attend_tree(*args, **dict(dict(out=q), **kw))
