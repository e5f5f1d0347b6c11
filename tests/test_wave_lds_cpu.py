"""LDS that a wave's lanes write for each other without a barrier: the compiler
sees each lane's addresses by themselves and may move a read of another lane's value
across the write. In the kernels' sources such a write is followed by
lanes_meet() (glu_core.hpp) before it is read, and the read by another before the same LDS
is written again."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp32_gemm_tuning_amd", "csrc")


def _kernel(file, name):
    """The text of a kernel, from its name to the next line that closes a scope at the margin."""
    text = open(os.path.join(CSRC, file)).read()
    at = re.search(rf"void (?:__launch_bounds__\([^)]*\) )?{name}\(", text).start()
    return text[at:text.index("\n}\n", at)]


def _in_order(text, *parts):
    """Whether the parts follow each other in the text, the first of them once."""
    assert text.count(parts[0]) == 1, parts[0]
    at = text.index(parts[0])
    for p in parts:
        at = text.find(p, at)
        if at < 0:
            return False
        at += len(p)
    return True


def test_lanes_meet_orders_memory():
    text = open(os.path.join(CSRC, "glu_core.hpp")).read()
    body = text[text.index("void lanes_meet() {"):]
    body = body[:body.index("}")]
    assert 'asm volatile("" ::: "memory");' in body and "__builtin_amdgcn_wave_barrier();" in body


def test_8_bit_rows_through_registers():
    k = _kernel("i8.hip", "k_i8_rows")
    assert _in_order(k, "fb.store(bv, ring", "lanes_meet();", "compute(ring);", "lanes_meet();", "\n        }")
