"""quantize_tokens computes rint(fl(x / s)) without a division.  This host test
compiles tests/token_quotient.c and checks that identity for every row maximum
and value up to a power of two; it needs no GPU."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_division_free_codes_round_like_ieee_division(tmp_path):
    exe = str(tmp_path / "token_quotient")
    subprocess.run(["gcc", "-O1", "-std=c99", "-ffp-contract=off", "-o", exe, os.path.join(HERE, "token_quotient.c"),
                    "-lm"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
