"""What the backward's tile kernel reads while the kernel before it may still write."""
import os
import re

from attention_attn_fwd_11_b200 import fa

SOURCE = os.path.join(os.path.dirname(os.path.abspath(fa.__file__)), "csrc", "bwd.cu")


def test_rows_of_the_row_kernel_are_not_read_as_constants():
    """The tile kernel starts before the row kernel has ended (a programmatic dependent launch), so LSE and D change
    during its lifetime: the read-only data path is not defined for them."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    assert "griddepcontrol.wait" in text
    written = re.findall(r"^\s*a\.(\w+)\[r\] = ", text, re.M)  # what bwd_prep_kernel stores for a row
    assert set(written) == {"nlse", "ndelta", "ext"}
    for name in written:
        assert not re.search(r"(__ldg|__ldcs|ld\.global\.nc)\s*\(?[^;\n]*\b%s\b" % name, text), name
