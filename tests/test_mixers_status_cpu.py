"""The status of operands that share memory."""
import weight_only_int4_w4a16_amd as w


def test_overlap_status_has_a_text():
    assert "share memory" in w.status_string(9) and w.status_string(9) != w.status_string(99)
