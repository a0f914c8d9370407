"""What the paged calls promise their callers, on the CPU: the text of a fault names everything that raises it, and
arguments whose memory a call would corrupt or misread are refused before anything is launched."""
import ctypes

import pytest
import torch

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


@pytest.mark.parametrize("T,H,token,head,overlap", [
    (4, 4, 0, 64, True), (4, 4, 256, 0, True), (4, 4, 64, 8, True), (4, 4, 248, 64, True), (4, 4, 64, 248, True),
    (2, 3, 128, 64, True), (3, 2, 64, 128, True), (4, 4, -256, 56, True), (5, 3, 104, 312, True),
    (4, 4, 256, 64, False), (4, 4, 64, 256, False), (4, 4, -256, 64, False), (1, 4, 0, 64, False), (4, 1, 64, 0, False),
    (1, 1, 0, 0, False), (2, 3, 64, 128, False), (3, 2, 128, 64, False), (2, 2, 72, 1000, False)])
@pytest.mark.parametrize("scale", [1, 2])
def test_rotated_queries_that_share_memory_are_refused(lib, scale, T, H, token, head, overlap):
    """Rows of the rotated queries that overlap would be written by several warps at once.  (Latent rows turn 64 columns,
    others hold 128.  A call whose strides pass goes on to the device, and fails here for want of one.)"""
    rows = [range(t * token + h * head, t * token + h * head + 64) for t in range(T) for h in range(H)]
    touched = [e for r in rows for e in r]
    assert (len(set(touched)) < len(touched)) == overlap  # the case is what it says
    if not overlap and torch.cuda.is_available():
        pytest.skip("the made-up pointers would reach a device")
    fn, width = ((lib.mla_cache_append, 64), (lib.mha_cache_append, 128))[scale - 1]
    kw = dict(B=1, T=T, H=H, cu_tokens=0, q_in=16, q_out=16, q_in_token_stride=width * H, q_in_head_stride=width,
              q_out_token_stride=token * scale, q_out_head_stride=head * scale, v_token_stride=width)
    got = fn(packed(**kw), None)
    assert got == 1 if overlap else got not in (0, 1, 2)
