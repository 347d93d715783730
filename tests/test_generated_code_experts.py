"""The experts' products issue their loads through the inline assembly of the two-group kernels (and its
non-temporal form), so the rule on M0 holds for them too: nothing else in these kernels reads or writes it."""
from test_generated_code import _functions, check_m0, code_objects  # noqa: F401  (a fixture)


def test_m0_checker_takes_the_streamed_load():
    good = ["s_mov_b32 m0, s2", "s_nop 0", "buffer_load_dwordx4 v1, s[8:11], s3 offen nt lds"]
    assert check_m0(good) == []
    assert len(check_m0(good[1:])) == 1
    assert len(check_m0(good + ["s_mov_b32 s1, m0"])) == 1


def test_grouped_kernels_use_m0_only_for_their_loads(code_objects):  # noqa: F811
    checked = {"grouped_kernel": 0, "grouped_pp_kernel": 0}
    streamed = 0
    for elf in code_objects:
        for name, ins in _functions(elf).items():
            kind = next((k for k in checked if k + "I" in name), None)  # I: template arguments follow
            if kind is None:
                continue
            text = [i for _, i, _ in ins]
            loads = [i for i in text if i.startswith("buffer_load") and i.endswith(" lds")]
            assert loads, name
            streamed += any(i.endswith(" nt lds") for i in loads)
            assert check_m0(text) == [], (name, check_m0(text)[:5])
            checked[kind] += 1
    # two input types x three output types, of three forward, three grad A and one grad B forms, and of the
    # two-group kernel's three modes
    assert checked == {"grouped_kernel": 6 * 7, "grouped_pp_kernel": 6 * 3}, checked
    assert streamed == 6 * 2, streamed  # the longer ring of 32-row tiles, forward and grad A
