"""What ``SpecVerifier.run_hidden`` refuses among its penalties, in front of any launch: no GPU is needed."""
from __future__ import annotations

import pytest
import torch

import speculative_decoding_verification_online_gb300 as sv


def verifier(k, V):
    v = object.__new__(sv.SpecVerifier)
    v.k, v.V, v.device, v.handle = k, V, torch.device("cuda", 0), None
    return v


@pytest.mark.parametrize("name", ["masks", "target_mask", "draft_masks", "mask_rows", "temperature", "history_lens"])
def test_names_that_are_none_are_refused(name):
    B, k, V, H = 2, 3, 40, 16
    pen = dict(history=torch.zeros(B, 4, dtype=torch.int32), history_len=torch.zeros(B, dtype=torch.int32))
    pen[name] = torch.zeros(B * (k + 1), 2, dtype=torch.int32)
    with pytest.raises(TypeError, match=name):
        verifier(k, V).run_hidden(torch.zeros(B, k + 1, H), torch.zeros(V, H), torch.zeros(B, k, H), torch.zeros(V, H),
                                  torch.zeros(B, k, dtype=torch.int32), 1.0, penalties=pen)


def test_the_names_that_are_taken_reach_the_next_check():
    B, k, V, H = 2, 3, 40, 16
    pen = dict.fromkeys(("history", "history_len", "prompt_len", "repetition", "frequency", "presence", "bias", "mask", "mask_row",
                         "draft_mask", "draft_mask_row"))
    with pytest.raises((ValueError, TypeError), match="target_hidden"):
        verifier(k, V).run_hidden(torch.zeros(B, k + 1, H), torch.zeros(V, H), torch.zeros(B, k, H), torch.zeros(V, H),
                                  torch.zeros(B, k, dtype=torch.int32), 1.0, penalties=pen)
