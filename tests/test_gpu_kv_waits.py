"""The cache operators' waits, arrival counts and scratch: calls that end without an error code, the same bits every
time, and a call after one that gave up."""
import numpy as np
import pytest
import torch

from test_gpu_kv import Step, nv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,dt", [(64, "bf16"), (64, "f16"), (128, "bf16"), (128, "f16"), (256, "bf16"), (256, "f16")])
def test_long_walks_end_alike_and_without_an_error_code(nv, dim, dt):  # noqa: F811
    """Long lists of tiles in every tensor-core kernel, call after call: no wait of any role runs out (lanes that poll for
    themselves have to stay within a phase of one another), and the results repeat bit by bit."""
    s = Step(nv, 40, [700, 300], [2500, 100], 8, 4, dim, 64, dt)
    q, table, lengths, offsets = s.rows(8).cuda(), s.i32(s.table), s.i32(s.lengths), s.i32(s.offsets)
    first = nv.kv_attention(q, s.kv, table, lengths, q_offsets=offsets, max_q=700)
    for _ in range(200):
        again = nv.kv_attention(q, s.kv, table, lengths, q_offsets=offsets, max_q=700)
    assert torch.equal(first, again) and torch.isfinite(first).all()
    assert nv.take_device_error() == 0
