"""The build's check of the kernels that set m0 in inline assembly, on assembly text."""
from linear_amd import build

LOAD = "\ts_mov_b32 m0, s53\n\ts_nop 3\n\tbuffer_load_dwordx4 v1, s[4:7], 0 offen lds\n"


def test_only_the_inline_loads_may_use_m0():
    assert build._other_m0_uses("kernel:\n\tv_mov_b32_e32 v0, 0\n" + LOAD + "; m0 in a comment\n" + LOAD) == []
    for other in ("\tds_gws_barrier v0 offset:0\n\ts_add_u32 m0, m0, 16\n", "\ts_mov_b32 s3, m0\n",
                  "\ts_mov_b32 m0, s2\n\tv_movrels_b32_e32 v0, v1\n",
                  "\ts_mov_b32 m0, s2\n\ts_nop 0\n\tbuffer_load_dword v1, s[4:7], 0 offen lds\n"):
        assert len(build._other_m0_uses(LOAD + other + LOAD)) == 1
    assert build._other_m0_uses("\ts_mov_b32 m0, s2\n") == ["s_mov_b32 m0, s2"]
