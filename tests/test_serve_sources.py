"""Rules that the sources of the norm-and-rotation and cache kernels keep, checked on their text (CPU)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "flashattention_backward_fa_gb300",
                    "csrc")


def _code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def _chained():
    """Files whose kernels may begin while the kernel that writes their inputs still runs, and the header
    that they share."""
    names = [n for n in sorted(os.listdir(CSRC)) if n.endswith(".cu") and "launch_chained(" in _code(n)]
    assert {"kernels_rope.cu", "kernels_kv8.cu", "kernels_kv8_attn.cu"} <= set(names)
    return names + ["rope_common.cuh"]


def test_no_read_only_loads_in_kernels_that_overlap_their_producers():
    """ld.global.nc is for memory that nothing writes during the kernel's lifetime, which begins before the
    kernel in front has ended."""
    for name in _chained():
        code = _code(name)
        for word in (r"__ldg\s*\(", r"ld\.global(\.\w+)*\.nc", r"__restrict__"):
            assert not re.search(word, code), (name, word)


def test_kernels_wait_before_they_read():
    """Every kernel of these files waits for the kernel in front, in its own body and before its loads."""
    for name in _chained()[:-1]:
        kernels = re.findall(r"__global__ void [^{]*?(\w+)\(const __grid_constant__ \w+ p\) \{(.*?)\n\}", _code(name),
                             flags=re.S)
        assert kernels, name
        for kernel, body in kernels:
            before, wait, _ = body.partition("wait_for_previous();")
            assert wait, kernel
            assert not re.search(r"__ld|_async\(|key_range\(|new_tokens\(|stage_weights|sequence_of\(", before), kernel
