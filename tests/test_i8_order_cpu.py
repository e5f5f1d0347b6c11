"""Of two bad arguments the norm's and the 8-bit entry points report the one that
stands first in the header's list of codes: every pair of the bad values of
test_i8_cpu.py, at every entry point (nothing is launched)."""
import re

import pytest

pytest.importorskip("torch")
import fp32_gemm_tuning_amd as sg  # noqa: E402
from test_i8_cpu import BAD, HEADER  # noqa: E402


def listed_codes():
    """The codes of the header's list, in its order."""
    text = open(HEADER).read()
    text = text[text.index("Return codes:"):text.index("A pointer is checked")]
    found = [sg.ERR_WORKSPACE if "WORKSPACE" in c else sg.ERR_TOO_LARGE if "TOO_LARGE" in c else int(c)
             for c in re.findall(r"(?<=[ *])(-\d+(?= )|SGEMM_F32_ERR_\w+)", text)]
    assert len(found) == len(set(found))
    return found


def test_the_list_holds_every_code():
    codes = {code for _, _, bad in BAD for *_, code in bad}
    assert codes <= set(listed_codes()) and len(listed_codes()) >= 31


@pytest.mark.parametrize("entry,good,bad", BAD, ids=[e.__name__ for e, _, _ in BAD])
def test_the_first_of_two_bad_arguments_is_reported(entry, good, bad):
    order = {c: i for i, c in enumerate(listed_codes())}
    wrong = []
    for i, (name, value, code) in enumerate(bad):
        for other, second, code2 in bad[i + 1:]:
            if other == name or "workspace" in name and "workspace" in other:
                continue
            first = min(code, code2, key=order.__getitem__)
            got = entry(*dict(good, **{name: value, other: second}).values(), stream=0)
            if got != first:
                wrong.append((name, value, other, second, got, first))
    assert not wrong


@pytest.mark.parametrize("size", ["M", "K"])
def test_a_size_too_large_comes_before_the_workspace(size):
    entry, good, _ = next(b for b in BAD if b[0] is sg.sgemm_f32_rms_norm_bwd)
    args = {k: 1 << 40 if k.startswith("ld") else v for k, v in good.items()}
    args[size] = (1 << 30) + 1
    assert entry(*dict(args, workspace=0, workspace_bytes=0).values(), stream=0) == sg.ERR_TOO_LARGE
