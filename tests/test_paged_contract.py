"""What the paged calls promise their callers, on the CPU: the text of a fault names everything that raises it, and
arguments whose memory a call would corrupt or misread are refused before anything is launched."""
from mla_decode_attention_11_b200 import binding as M


def test_fault_texts_name_every_cause():
    """Codes 7 and 8 come from decodes (clamped, or read as zeros) and from appends (a token skipped, or its row not
    written): a caller must not read that the value was clamped and the data written."""
    length, page = M.status_string(7), M.status_string(8)
    assert "clamped" in length and "rotation table" in length and "skipped" in length
    assert "block-table entry" in page and "read as zeros" in page and "not written" in page
