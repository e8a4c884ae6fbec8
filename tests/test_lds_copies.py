"""Wait states in front of the copies from buffers into LDS: the check itself, and the built library (no GPU)."""
import os

import pytest

from exact_int8_gemm_amd import build, wait_states


def test_copies_into_lds_keep_their_wait_states():
    if not os.path.exists(build.LIB):
        build.build_library()
    copies, wrong = wait_states.check(build.LIB, build.OBJDUMP, build.ARCH)
    assert copies > 1000                            # the tiled kernels' copies were seen
    assert not wrong, "%d of %d copies come too early, the first: %r" % (len({w[:2] for w in wrong}), copies, wrong[0])


def listing(*lines):
    return "0000 <f>:\n" + "\n".join("\t%s // %012X: 0 %s" % (l.partition("@")[0], 4 * n, l.partition("@")[2])
                                     for n, l in enumerate(lines))


COPY = "buffer_load_dwordx4 v0, s[4:7], 0 offen lds"


@pytest.mark.parametrize("lines,wrong", [
    (["v_readlane_b32 s6, v9, 1", "s_mov_b32 m0, s1", "s_nop 3", COPY], 0),
    (["v_readlane_b32 s6, v9, 1", "s_mov_b32 m0, s1", "s_nop 2", COPY], 1),
    (["v_readfirstlane_b32 s4, v9", "s_nop 4", "buffer_load_dword v0, s[4:7], s8 offen lds"], 0),
    (["v_readfirstlane_b32 s8, v9", "s_nop 3", "buffer_load_dword v0, s[4:7], s8 offen lds"], 1),
    (["v_readlane_b32 s8, v9, 1", "s_mov_b32 m0, s1", "s_nop 0", COPY], 0),
    (["s_mov_b32 m0, s1", COPY], 1),
    (["s_mov_b32 s5, s1", "s_nop 0", COPY], 0),
    (["v_cmp_lt_u32_e64 s[6:7], v1, v2", "s_nop 0", COPY], 1),
    (["v_add_co_u32_e64 v1, s[6:7], v1, v2", "s_nop 0", COPY], 1),
    (["v_add_u32_e32 v1, s6, v1", "s_nop 0", COPY], 0),
    (["v_readlane_b32 s8, v9, 1", "buffer_load_dwordx4 v[0:3], v4, s[4:7], 0 offen"], 0),
    (["s_mov_b32 m0, s1", "buffer_load_dword v0, s[4:7], 0 offen offset:64 lds sc0"], 1),
    (["v_readlane_b32 s2, v9, 1", "s_nop 3", "global_load_lds_dwordx4 v0, s[2:3]"], 1),
    # over a branch: the write in front of the jump back, and one that no path leads on from
    (["s_nop 7", "s_nop 0", COPY, "s_nop 7", "v_readlane_b32 s4, v9, 1", "s_cbranch_scc0 9@<f+0x4>"], 1),
    (["s_branch 9@<f+0xc>", "v_readlane_b32 s4, v9, 1", "s_endpgm", COPY], 0)])
def test_the_check_itself(lines, wrong):
    code = wait_states.parse(listing(*lines))["f"]
    copies, found = wait_states.too_early(code)
    assert copies == sum(" lds" in l or "_lds_" in l for l in lines) and len(found) == wrong
