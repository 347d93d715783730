"""The microscaled products load codes in pieces of 16 bytes and scales in dwords through the inline assembly that writes M0 in
front of each load to LDS. The compiler does not know that, so nothing else in these kernels may read or write M0."""
from test_generated_code import IMPLICIT_M0, _functions, code_objects  # noqa: F401  (a fixture)
import re

LOAD = re.compile(r"buffer_load_dword(x4)? .* lds$")


def violations(instructions):
    bad = []
    for i, ins in enumerate(instructions):
        op = ins.split()[0]
        if IMPLICIT_M0.match(op):
            bad.append(f"{i}: {ins} uses M0 implicitly")
        elif re.search(r"\bm0\b", ins):
            if not ins.startswith("s_mov_b32 m0,") or instructions[i + 1:i + 2] != ["s_nop 0"] or not any(
                    LOAD.match(x) for x in instructions[i + 2:i + 3]):
                bad.append(f"{i}: {ins} is not a write, one wait state and a load to LDS")
        elif op.startswith("buffer_load") and ins.endswith(" lds"):
            if not LOAD.match(ins) or i < 2 or instructions[i - 1] != "s_nop 0" or not instructions[i - 2].startswith("s_mov_b32 m0,"):
                bad.append(f"{i}: {ins} has no M0 write of its own in front of it")
    return bad


def test_violations_of_each_kind_are_found():
    good = ["s_mov_b32 m0, s2", "s_nop 0", "buffer_load_dword v1, s[8:11], s3 offen lds", "s_mov_b32 m0, s2", "s_nop 0",
            "buffer_load_dwordx4 v1, s[8:11], s3 offen nt lds", "s_endpgm"]
    assert violations(good) == []
    assert len(violations(good[:1] + good[2:])) == 2                              # wait state missing
    assert len(violations(good[1:])) == 1                                         # load without its own M0 write
    assert len(violations(good[:2])) == 1                                         # write without its load
    assert len(violations(good + ["s_add_u32 s5, m0, 4"])) == 1                   # the compiler reading M0
    assert len(violations(good + ["s_sendmsg sendmsg(MSG_DEALLOC_VGPRS)"])) == 1  # implicit use


def test_products_use_m0_only_for_their_loads(code_objects):  # noqa: F811
    checked = {"mx_tile_kernel": 0, "mx_skinny_kernel": 0, "mx_pp_kernel": 0}
    dwords = 0
    for elf in code_objects:
        for name, ins in _functions(elf).items():
            kind = next((k for k in checked if k + "I" in name), None)  # I: template arguments follow
            if kind is None:
                continue
            text = [i for _, i, _ in ins]
            assert violations(text) == [], (name, violations(text)[:5])
            loads = [i for i in text if LOAD.match(i)]
            assert loads or kind == "mx_skinny_kernel", name
            dwords += any(i.startswith("buffer_load_dword ") for i in loads)
            checked[kind] += 1
    # five forms (three formats, and the two with bf16 instructions) of three and two tiles; three formats by three result types,
    # which load scales in dwords
    assert checked == {"mx_tile_kernel": 5 * 3, "mx_skinny_kernel": 5 * 2, "mx_pp_kernel": 3 * 3}, checked
    assert dwords == 9, dwords
