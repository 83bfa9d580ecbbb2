"""Host check of the division behind the AdamW step's 8-bit moments: its codes are those of the correctly rounded
quotient next to every border between two codes, over the range of the scales.  Compiled with the host gcc."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    out = str(tmp_path_factory.mktemp("quot") / "moment_quotient_check")
    subprocess.run([gcc, "-O2", "-mfma", "-ffp-contract=off", "-o", out, os.path.join(HERE, "moment_quotient_check.c"), "-lm"],
                   check=True)
    return out


def _run(exe, *args):
    r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, check=True)
    return tuple(map(int, r.stdout.split()))


@pytest.mark.parametrize("emin,emax", [(-126, -100), (-100, -60), (-60, 0), (0, 127)])
def test_codes_of_the_rounded_quotient(checker, emin, emax):
    n, bad_m, bad_v = _run(checker, emin, emax, 500, 0)
    assert n > 1_000_000 and bad_m == 0 and bad_v == 0


def test_small_scales_need_the_power_of_two(checker):
    # the remainder underflows: why scales below 2^-60 are moved up
    _, bad_m, bad_v = _run(checker, -126, -100, 500, 1)
    assert bad_m > 0 and bad_v > 0
