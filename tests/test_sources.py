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


def test_a_dependent_grid_waits_before_it_ends():
    """A kernel that starts while the one before it still runs must not end
    without having waited for it: what follows on the stream, or in a captured
    graph, waits for this kernel alone. So no plain return stands before the wait,
    and where rows leave early they do it by leave_merge, which waits."""
    waits, launched = {}, set()
    for f in sorted(CSRC.glob("*.cu")):
        text = re.sub(r"//[^\n]*", "", f.read_text())
        for part in re.split(r"__global__", text)[1:]:
            name = re.search(r"(\w+_kernel)\s*\(", part).group(1)
            at = part.find('"griddepcontrol.wait')
            waits[name] = part[:at] if at >= 0 else None
        if "ProgrammaticStreamSerialization" in text:
            launched |= set(re.findall(r"cudaLaunchKernelEx\(&\w+,\s*(\w+_kernel)", text))
    assert {"merge_kernel", "prefix_merge_kernel", "decode_pair_kernel", "compact_move_kernel"} <= launched
    for name in launched:
        assert waits[name] is not None, name
        assert not re.search(r"\breturn\s*;", waits[name]), name
    leave = re.search(r"void leave_merge\(\) \{(.*?)\n\}", (CSRC / "merge_row.cuh").read_text(), re.S).group(1)
    assert re.search(r"if \(blockIdx\.x == 0\)\s*asm volatile\(\"griddepcontrol\.wait", leave)


def test_no_launch_has_a_number_of_sms_written_into_it():
    """Grids follow the device's own count (152 here, and its small multiples)."""
    for f in sorted(CSRC.glob("*.cu")):
        code = re.sub(r"//[^\n]*", "", f.read_text())
        assert not re.search(r"\b(76|152|304|456|608|912|1216)\b", code), f.name
