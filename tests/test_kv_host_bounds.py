"""Host-side bounds of the attention call: a line of work that its blocks could
not count is refused before the device is touched."""
import pytest

import rotation_post_quantization_b200 as rq

A = 0x10000   # a fake, aligned device address: never dereferenced


def attention(B, N, max_pages, page_size=128, kv_heads=1024, q_heads=1024, ws_bytes=0):
    c = rq._KvCacheC(A, A, A, A, 4, page_size, kv_heads, 64)
    b = rq._KvBatchC(A, A, A, B, max_pages, N)
    ld = q_heads * 64
    return rq.lib.respin_kv_attention(c, b, A, q_heads, ld, 0, 1, 0, 0.125, A, ld, None, A, ws_bytes, None)


@pytest.mark.parametrize("B,N,max_pages", [(65536, 65536, 1 << 13), (65536, 65536, (1 << 24) - 512), (64, 1 << 20, (1 << 24) - 512)])
def test_line_of_work_beyond_its_count(B, N, max_pages):
    # (a workspace of no bytes would be refused next)
    assert attention(B, N, max_pages, ws_bytes=0) == rq.RESPIN_ERR_UNSUPPORTED and "2^38" in rq.last_error()


@pytest.mark.parametrize("B,N,max_pages", [(65536, 65536, 1 << 10), (64, 1 << 20, 1 << 13), (1, 1, (1 << 24) - 512)])
def test_large_but_countable_lines_are_taken(B, N, max_pages):
    assert attention(B, N, max_pages, ws_bytes=0) == rq.RESPIN_ERR_INVALID_ARG and "workspace" in rq.last_error()
