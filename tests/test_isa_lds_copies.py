"""The kernels copy global memory into LDS with inline assembly: a copy takes
its LDS address from m0, which a scalar instruction writes just before.  On
gfx950 such a copy needs one wait state after a scalar write of m0 (without it
the copy may land at the address of the one before), and the compiler, which
does not look into the assembly, adds none.  This test checks the assembly
text of every source.
"""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_gemv_amd", "csrc")


def copies(source):
    """(copies into LDS, those right after a scalar write of m0, those whose m0 the same block does not write) in the inline
    assembly of a source."""
    n = close = foreign = 0
    for block in re.findall(r'\basm\s+volatile\s*\(\s*((?:"(?:[^"\\]|\\.)*"\s*)+)', source):
        text = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', block))
        ins = [i.strip() for i in re.split(r"\\n(?:\\t)?", text) if i.strip()]
        for i, op in enumerate(ins):
            if re.match(r"(global_load_lds|buffer_load\w* .*\blds$)", op):
                n += 1
                wrote = [bool(re.match(r"s_\w+ m0,", p)) for p in ins[:i]]
                close += bool(wrote and wrote[-1])
                foreign += not any(wrote)
    return n, close, foreign


def test_scanner_finds_planted_hazards():
    near = r'''asm volatile("s_mov_b32 m0, %1\n\t"
                 "global_load_lds_dwordx4 %0, off" ::"v"(p), "s"(at) : "memory");'''
    assert copies(near) == (1, 1, 0)
    assert copies(near.replace(r'%1\n\t"', r'%1\n\ts_nop 0\n\t"')) == (1, 0, 0)
    assert copies(r'asm volatile("s_add_u32 m0, m0, 16\n\tbuffer_load_dword %0, %1, 0 offen lds" :: "v"(a), "s"(b));') == (1, 1, 0)
    assert copies(r'asm volatile("global_load_lds_dword %0, off" ::"v"(p));') == (1, 0, 1)
    assert copies(r'asm volatile("s_mov_b32 m0, %1\n\tglobal_load_dword %0, %2, off" : "=v"(v));') == (0, 0, 0)


def test_every_copy_into_lds_waits_for_m0():
    found = {os.path.basename(p): copies(open(p).read()) for p in sorted(glob.glob(os.path.join(CSRC, "*.h*")))}
    assert found["moe_lds.hpp"][0] >= 1 and found["moe_matmul_i8.hip"][0] >= 2
    assert all(close == 0 and foreign == 0 for _, close, foreign in found.values()), {k: v for k, v in found.items() if v[0]}
    # the mnemonic nowhere else, such as in a macro that the above does not see
    for p in sorted(glob.glob(os.path.join(CSRC, "*"))):
        if os.path.isfile(p):
            assert len(re.findall(r"global_load_lds_\w+ %", open(p).read())) == found.get(os.path.basename(p), (0,))[0], p
