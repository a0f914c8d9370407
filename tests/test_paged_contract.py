"""What the paged calls promise their callers, on the CPU: the text of a fault names everything that raises it, and
arguments whose memory a call would corrupt or misread are refused before anything is launched."""
import ctypes

import pytest

from mla_decode_attention_11_b200 import binding as M
from tests.test_paged_boundary import FIELDS

OK = dict(B=2, T=4, H=0, Hkv=1, rope_dim=64, interleaved=0, num_positions=100, page_size=16, num_pages=4, table_width=4,
          table_stride=4, cu_tokens=16, seqlens=16, block_table=16, cos_sin=16, k=16, v=16, q_in=0, q_out=0, k_pages=16,
          v_pages=16, k_token_stride=512, k_head_stride=0, v_token_stride=64, v_head_stride=0, q_in_token_stride=0,
          q_in_head_stride=0, q_out_token_stride=0, q_out_head_stride=0, status=0, kv_scale=0.0, reserved=0)


@pytest.fixture(scope="module")
def lib():
    return M.load_library()


def packed(**kw):
    assert set(kw) <= set(OK)
    a = {**OK, **kw}
    return M._APPEND.pack(*(a[f] for f in FIELDS))


def test_fault_texts_name_every_cause():
    """Codes 7 and 8 come from decodes (clamped, or read as zeros) and from appends (a token skipped, or its row not
    written): a caller must not read that the value was clamped and the data written."""
    length, page = M.status_string(7), M.status_string(8)
    assert "clamped" in length and "rotation table" in length and "skipped" in length
    assert "block-table entry" in page and "read as zeros" in page and "not written" in page


def test_append_behind_a_prefix_rejects(lib):
    """The prefix's length is a device pointer, never absent, and the rest is checked as without one."""
    call = lambda prefix, **kw: lib.mla_cache_append_prefix(packed(**kw), ctypes.c_void_p(prefix), None)
    assert call(0) == 1 and call(18) == 2
    assert call(16, B=0) == 1 and call(16, cos_sin=8) == 2
    assert call(16, T=0, k=0, v=0) == 0  # nothing to do
    assert lib.mla_cache_append_prefix(None, ctypes.c_void_p(16), None) == 1
