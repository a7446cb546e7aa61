"""The operators around a tree's target pass called by several host threads at once."""
from __future__ import annotations

import threading

import pytest
import torch

from tests.test_gpu_step_operators import sv  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def test_penalties_of_different_sizes_from_several_threads(sv):
    # One kernel with 80 KB of shared memory (with biases) and with 48 KB, launched from four threads.  All sequences are padded
    # ones, so that the host's part is what takes the time; only the status counts.
    V, B = 65536, 40
    logits = torch.zeros(B, V, dtype=torch.bfloat16, device="cuda")
    history = torch.zeros(B, 4, dtype=torch.int32, device="cuda")
    padded = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    zeros = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    values = torch.zeros(4, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(4)]
    call = sv.load().spec_verify_penalties
    refused = [None] * 4

    def work(i):
        biases = (zeros.data_ptr(), zeros.data_ptr(), values.data_ptr(), 4) if i % 2 else (None, None, None, 0)
        args = (logits.data_ptr(), 1, V, logits.data_ptr(), 1, V, V, history.data_ptr(), 4, 4, padded.data_ptr(), None,
                None, None, zeros.data_ptr(), B, 0, 0, None, None, None, *biases, None, 0, 0, None, 0, streams[i].cuda_stream)
        refused[i] = sum(call(*args) != 0 for _ in range(20000))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0] * 4
    assert not bool(logits.any())
