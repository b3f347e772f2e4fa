"""Rules that no run can show broken, read from the sources of the fine-tuning operators
(layernorm.cu, seqloss.cu, gradclip.cu)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "spectral_corrected_optimizer_gb300", "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def kernel(name, text):
    return re.search(r"__global__ void[^;{]*\b%s\([^{]*\{(.*?)\n\}\n" % name, text, re.S).group(1)


def test_a_ring_that_gives_up_a_wait_lets_its_copies_end():
    # Shared memory that a copy still writes to belongs, after the block has left, to the next block of the SM.
    body = kernel("layernorm_backward_kernel", source("layernorm.cu"))
    loop = body[body.index("for (int64_t tile = 0"):]
    # one wait, and no copy is asked for once it gave up
    assert "ok = ok && (mbar_wait_bounded(&full[stage], phase, flag, 0x701u) || give_up());" in loop
    assert loop.count("mbar_wait") == 1 and loop.count("ok = ") == 1 and "bool ok = true;" in body
    assert re.findall(r"if \(([^\n]*)\) fetch\(tile \+ a\.stages, stage\);", loop) == ["tid == 0 && ok && tile + a.stages < tiles"]
    assert loop.count("fetch(") == 1
    # the thread that asked for them waits, with a limit, for both phases of every barrier: one of them is the phase that a
    # copy under way completes, the other is complete already or holds the thread up to the limit
    drain = re.search(r"auto give_up = \[&\] \{\s*if \(tid == 0\)\s*for \(int i = 0; i < 2 \* a\.stages; \+\+i\) "
                      r"mbar_wait_limit\(&full\[i / 2\], i & 1, nullptr, 0u, kDrainLimit\);\s*return false;\s*\};", body)
    assert drain and body.count("mbar_wait") == 2 and "if (tid == 0)\n        for (int i = 0; i < a.stages && i < tiles; ++i) fetch(i, i);" in body


def test_kernels_that_wait_for_the_launch_in_front_read_it_with_plain_loads():
    # as test_stage_ends_sources.py has it for the others; what these read with __ldg are inputs of the call, complete
    # before its first, ordinary launch
    for name in ("layernorm.cu", "seqloss.cu", "gradclip.cu"):
        text = source(name)
        kernels = re.findall(r"__global__ void([^;{]*)\{(.*?)\n\}\n", text, re.S)
        waiting = [(head, body) for head, body in kernels if "grid_dependency_wait()" in body]
        assert len(kernels) >= 3 and waiting, name
        for head, body in waiting:
            assert not re.search(r"const [\w ]+\*\s*__restrict__", head), (name, head)
            assert "__ldg" not in body and ".nc." not in body, (name, head)
        assert set(re.findall(r"__ldg\(([\w.]+)", text)) <= {"a.mean", "a.rstd"}, name
        assert "kLasting" not in text, name
