"""Caches whose strides put entries or scales over one another are refused by the calls that write them: their threads would
write one place at once.  The calls name a device that does not exist, so that nothing runs."""
from __future__ import annotations

import pytest

import speculative_decoding_verification_online_gb300 as sv
from speculative_decoding_verification_online_gb300 import spec_verify as m
from tests.test_step_operators_refusals import ATTEND, KEEP, WRITE, _cached, library  # noqa: F401  (library is a fixture)

NO_DEVICE = 1 << 20
LAYERS = dict(layers=3, layer_stride=9 * 4096, scale_layer_stride=9 * 4 * 2)


@pytest.mark.parametrize("cache,apart", [
    ({}, True), (dict(page_stride=4096 - 16), False), (dict(page_stride=64), False), (dict(head_stride=1024 - 64), False),
    (dict(head_stride=64, token_stride=256), True),  # heads inside of tokens
    (dict(head_stride=48, token_stride=256), False), (dict(head_stride=64, token_stride=256 - 64), False),
    (dict(page_stride=8192, head_stride=2048, token_stride=128), True),  # keys and values side by side
    (dict(pages=1, page_stride=0), True), (dict(pages=1, heads=1, page_stride=16, head_stride=16), True),
    (dict(head_stride=1024 * 9, page_stride=1024), True)])  # heads outside of pages
def test_entries(cache, apart):
    want = m.SV_ECUDA if apart else m.SV_EINVAL
    assert _cached(sv.spec_verify_cache_write, WRITE, dict(device=NO_DEVICE), cache) == want
    assert _cached(sv.spec_verify_cache_keep, KEEP, dict(device=NO_DEVICE), cache) == want


@pytest.mark.parametrize("cache,apart", [
    ({}, True), (dict(scale_layer_stride=0), False), (dict(scale_layer_stride=71), False), (dict(layer_stride=9 * 4096 - 16), False),
    (dict(layer_stride=64, token_stride=64 * 3, head_stride=4096, page_stride=16384), True), (dict(layers=1, scale_layer_stride=0), True)])
def test_layers(cache, apart):
    assert _cached(sv.spec_verify_cache_keep, KEEP, dict(device=NO_DEVICE), dict(LAYERS, **cache)) == (
        m.SV_ECUDA if apart else m.SV_EINVAL)


def test_a_call_that_only_reads_takes_them():
    assert _cached(sv.spec_verify_attend, ATTEND, dict(device=NO_DEVICE), dict(page_stride=64)) == m.SV_ECUDA
