"""Limits of the serving-side entry points at their edges, without a GPU: no test here enqueues GPU work."""
import ctypes

import pytest

import weight_only_int4_act_b200 as awq

FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced
SHAPE, WORKSPACE = 2, 3


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_context_ends_before_the_token_index_does(page):
    """Tables of 2^31 - 128 tokens or more are refused: the last tile's token indices would pass 31 bits. (The workspace is
    too small, so that a call which passes the shape checks stops there.)"""
    cfg = awq.make_kv4(4, 128, page)

    def call(pages):
        return awq.lib().awq_kv4_attention(FAKE, 0, 1024, 128, 1, 8, None, 1, FAKE, 9, FAKE, pages, FAKE, 1, 0.1,
                                           ctypes.byref(cfg), FAKE, None, FAKE, 0, None)
    most = (2 ** 31 - 1 - 128) // page
    assert call(most) == WORKSPACE
    assert most * page < 2 ** 31 - 128 <= (most + 1) * page
    for pages in (most + 1, 2 ** 31 // page):
        assert call(pages) == SHAPE
