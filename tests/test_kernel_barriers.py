"""The raw workgroup barrier is written in one place, with the compiler fence
that it needs (CPU only, from the kernels' sources).

The builtin emits s_barrier and is no memory operation to the compiler. The
waits in front of it keep memory operations above them; without a fence behind
it, a read of LDS that other wavefronts' DMA filled may be scheduled above the
barrier.
"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "token_dispatch_grouped_amd", "csrc")


def _sources():
    for f in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, f)) as fh:
            yield f, fh.read()


def test_every_raw_barrier_is_fenced():
    seen = 0
    for name, text in _sources():
        text = re.sub(r"//.*", "", text)
        for m in re.finditer(r"__builtin_amdgcn_s_barrier\(\);", text):
            seen += 1
            assert re.match(r'\s*asm volatile\("" ::: "memory"\);', text[m.end():]), (
                f"{name}:{text.count(chr(10), 0, m.start()) + 1}: no fence behind the barrier")
    assert seen == 1, "barrier() is the one place that emits it"
