"""CPU check of a rule in the products' source (nvfp4_gemm.hip): a stage's place
in LDS is refilled by copies that the compiler does not see, issued by other waves
once a barrier has passed. So a wave's reads have to have returned before it
arrives there, and the source has to say so: the bare barrier instruction only
stands behind a wait for LDS reads. (Today's code would run right without it, as
the compiler uses every read before the barrier; nothing holds it to that.)"""
import os
import re

import block_scaled_fp4_gemv_amd as g


def source():
    text = open(os.path.join(g.PKG_DIR, "csrc", "nvfp4_gemm.hip")).read()
    return re.sub(r"//[^\n]*", "", text)


def test_barriers_wait_for_lds_reads():
    text = source()
    bare = [m.start() for m in re.finditer(r"__builtin_amdgcn_s_barrier\s*\(|\bs_barrier\b", text)]
    assert bare, "no barrier found: the check looks for the wrong name"
    for at in bare:
        before = text[:at].rstrip().split(";")[-2]          # the statement before
        assert re.search(r"asm\s+volatile\s*\(\s*\"s_waitcnt lgkmcnt\(0\)\"\s*:\s*:\s*:\s*\"memory\"\s*\)", before), before


def test_wave_ring_waits_before_it_refills():
    """The wave kernel has no barrier in its loop: the wait stands before the copies."""
    loop = source().split("nvfp4_gemm_wave_kernel")[1].split("for (; n + NS - 1 < stages; ++n)")[1]
    assert loop.index('"s_waitcnt lgkmcnt(0)"') < loop.index("issue(n + NS - 1")
