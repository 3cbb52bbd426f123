"""A kernel that is launched early (programmatic stream serialisation) runs while the kernel ahead of
it still writes. What that one writes is not constant for this one's lifetime, so it may not be
loaded as if it were: not by __ldg, and not through a pointer to const that is __restrict__, which
lets the compiler take the same load and move it ahead of grid_dependency_wait(). No run shows the
difference while the compiler leaves such loads where they stand, so the source is checked."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "moe_expert_grouped_gb300", "csrc")

# kernel, and the names by which it reads what the kernel ahead of it writes
READ = [
    ("gg_permute.cu", "permute_scatter_kernel", ["block_hist"]),
    ("gg_permute.cu", "scatter_rows_kernel", ["row_of_slot", "pad_slot_of_row", "offsets"]),
    ("gg_mx_quant.cu", "quantize_scatter_kernel", ["tb"]),
    ("gg_route.cu", "route_finalise_kernel", ["part_p", "part_n", "part_z"]),
    ("gg_gemm_f8.cu", "f8_gemm_kernel", ["s"]),
    ("gg_adamw.cu", "norm_join_kernel", ["partial"]),
]


def _text(path, name):
    with open(os.path.join(CSRC, path)) as f:
        src = re.sub(r"//[^\n]*", "", f.read())
    start = re.search(name + r"\s*\(\s*const", src).start()
    end = src.find("__global__", start)
    return src[start:end if end > 0 else len(src)]


@pytest.mark.parametrize("path,name,read", READ, ids=[n for _, n, _ in READ])
def test_what_the_kernel_ahead_writes_is_not_read_as_constant(path, name, read):
    text = _text(path, name)
    assert "grid_dependency_wait()" in text
    for pointer in read:
        assert re.search(r"\b%s\b" % pointer, text)
        assert not re.search(r"__ldg\(\s*%s\b" % pointer, text)
        assert not re.search(r"const\s+\w+\*\s*__restrict__\s+%s\b" % pointer, text)
