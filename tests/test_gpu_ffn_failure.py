"""Failure detection of the gated block's kernels without a fault: bounded device waits that
run out.

With the limit below zero every main wait gives up at its first unsuccessful poll. The kernel
drains its copies and products, frees its tensor memory, sets the sticky error word and exits;
the word is read and cleared, and the next call's results are the usual ones: the context
stays usable. A CTA pair (more than 128 tokens) mirrors the give-up into its other CTA; a
cluster of the few-token form meets at its barriers. (A pair's poll itself waits for a while: its
sizes are such that a tile's products take longer.)
"""
import ctypes

import pytest
import torch

import gpu_util as gu
from test_gpu_ffn import normal

pytestmark = pytest.mark.gpu

ERR_TIMEOUT = 5
DEVERR_TIMEOUT = 0x4


@pytest.mark.parametrize("T,H,I", [(3, 2048, 512), (100, 1024, 1024), (300, 4096, 512), (2057, 2048, 3304)],
                         ids=["few", "few_128", "pairs", "several_tiles"])
def test_bounded_waits_give_up_and_recover(T, H, I):
    m = gu.need_gpu()
    dt = torch.bfloat16
    x, W1, dh = normal(1, (T, H), dt), normal(2, (2 * I, H), dt, 0.02), normal(3, (T, I), dt, 0.1)
    calls = (lambda: (m.moe_gated_ffn(x, W1),), lambda: m.moe_gated_ffn_backward(dh, x, W1))
    assert m.ffn_get_error() == 0
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        m.ffn_set_wait_limit(-1)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            m.ffn_set_wait_limit(0)
        word = ctypes.c_uint32(0)
        st = m.lib().moe_ffn_get_error(torch.cuda.current_stream().cuda_stream, ctypes.byref(word))
        assert st == ERR_TIMEOUT and word.value == DEVERR_TIMEOUT
        m.ffn_clear_error()
        assert m.ffn_get_error() == 0
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(call(), want))
        assert m.ffn_get_error() == 0
