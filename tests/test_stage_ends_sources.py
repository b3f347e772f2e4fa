"""A rule that no run can show broken, read from the stage-end operators' sources:
a read-only load (__ldg, or a const __restrict__ parameter, which the compiler
may read the same way) is for memory that nothing writes while the kernel is
resident.  A kernel that waits for the launch in front of it is resident while
that launch writes, and the helpers of rowvec.cuh serve such kernels, in-place
calls and sums that are added to."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "spectral_corrected_optimizer_gb300", "csrc")
KERNEL = re.compile(r"__global__ void(?P<head>[^;{]*)\{(?P<body>.*?)\n\}\n", re.S)


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def dependents():
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        for m in KERNEL.finditer(source(os.path.basename(path))):
            if "grid_dependency_wait()" in m["body"]:
                yield os.path.basename(path), m["head"], m["body"]


def test_kernels_that_wait_for_the_launch_in_front_read_it_with_plain_loads():
    found = list(dependents())
    assert len(found) >= 7  # the sort, sums and joins, dgamma, and the head's four
    for name, head, body in found:
        assert not re.search(r"const [\w ]+\*\s*__restrict__", head), (name, head)
        assert "__ldg" not in body and ".nc." not in body, (name, head)


def test_row_helpers_make_plain_loads_but_of_lasting_tensors():
    rowvec, embed = source("rowvec.cuh"), source("embed.cu")
    assert rowvec.count("__ldg") == 1 and "return LASTING ? __ldg(p) : *p;" in rowvec and "LASTING = true" not in rowvec
    assert "__ldg" not in embed
    # the one tensor that is read so: dy, which is complete before the gradient's first, ordinary launch
    for name in ("embed.cu", "resnorm.cu", "head_loss.cu", "head_gemm.cu"):
        uses = re.findall(r"load\w*<kLasting>\((\w+)", source(name))
        assert set(uses) <= {"dy"}, (name, uses)
    load_raw = re.search(r"load_raw\(.*?\n\}\n", source("resnorm.cu"), re.S)
    assert load_raw and "__ldg" not in load_raw.group(0)
