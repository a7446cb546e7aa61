"""Strides of dimensions of one entry, which mean nothing, are not looked at.  The calls name a device that does not exist: an
entry point that takes the arguments says so (``SV_ECUDA``), and nothing runs."""
from __future__ import annotations

import pytest
import torch

import speculative_decoding_verification_online_gb300 as sv
from speculative_decoding_verification_online_gb300 import spec_verify as m
from tests.test_step_operators_refusals import ATTEND, CACHE, _cached, library  # noqa: F401  (library is a fixture)

NO_DEVICE = 1 << 20


@pytest.mark.parametrize("change,heads,status", [
    (dict(B=1, total_nodes=0, q_row=515), 4, m.SV_ECUDA), (dict(B=1, total_nodes=0, q_row=3, q_head=68), 4, m.SV_EINVAL),
    (dict(q_row=515), 4, m.SV_EINVAL), (dict(q_heads=1, q_head=77), 1, m.SV_ECUDA), (dict(q_heads=2, q_head=77), 1, m.SV_EINVAL)])
def test_attend(change, heads, status):
    assert _cached(sv.spec_verify_attend, ATTEND, dict(change, device=NO_DEVICE), dict(heads=heads)) == status


def test_python_cache():
    # one page, one head and one layer: any strides of theirs, and different ones of k and of v
    f8 = torch.float8_e4m3fn

    def entries(page, head):
        return torch.zeros(16 * 64, dtype=torch.uint8).view(f8).as_strided((1, 1, 16, 64), (page, head, 64, 1))

    scales = [torch.zeros(2).as_strided((1, 1, 2), s) for s in ((2, 2, 1), (7, 5, 1))]
    c = m._cache((entries(1024, 1024), entries(17, 3), *scales), torch.device("cpu"), False)
    assert (c.pages, c.heads, c.page_tokens, c.block, c.dim) == (1, 1, 16, 8, 64) and c.token_stride == 64
    with pytest.raises(ValueError, match="strides"):
        wide = torch.zeros(16 * 80, dtype=torch.uint8).view(f8).as_strided((1, 1, 16, 64), (1024, 1024, 80, 1))
        m._cache((entries(1024, 1024), wide, *scales), torch.device("cpu"), False)
    assert CACHE["heads"] == 4


@pytest.mark.gpu
def test_attend_a_row_of_a_packed_buffer():
    from tests.test_gpu_step_operators import attend_case
    c = attend_case(6, [200], [0], 2, 3, 64, 32, 16)
    want = sv.attend_tree(**c)
    packed = torch.zeros(1, 6 * 64 + 3, dtype=torch.bfloat16, device="cuda")
    q = packed.as_strided((1, 6, 64), (6 * 64 + 3, 64, 1))
    q.copy_(c["q"])
    assert q.stride(0) % 8 and torch.equal(sv.attend_tree(**dict(c, q=q)), want)
