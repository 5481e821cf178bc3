"""What the CUDA sources may not hold, read as text."""
import pathlib
import re

CSRC = pathlib.Path(__file__).resolve().parent.parent / "paged_mla_decode_06_gb300" / "csrc"


def test_no_copy_is_multicast_to_a_cluster():
    """One library serves processes of one GPU and of several: its copies go to
    the issuing CTA alone."""
    files = sorted(CSRC.glob("*.cu")) + sorted(CSRC.glob("*.cuh"))
    assert len(files) > 10
    for f in files:
        # (adjacent string literals of an asm statement are one instruction)
        text = re.sub(r'"\s*"', "", f.read_text())
        assert not re.search(r"cp\.async\.bulk[^;]*multicast::cluster", text), f.name
