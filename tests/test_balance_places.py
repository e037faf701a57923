"""The places of the balance loss's partial sums, under AddressSanitizer and
UndefinedBehaviorSanitizer on the CPU: every sequence of drawn batches (empty ones, at
the last token too; none of the tokens in any; no tokens at all) finds the sums of its
own tokens, each once, and reads nowhere else.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FLAGS = ["-std=c++17", "-O1", "-g", "-Wall", "-fsanitize=address,undefined", "-fno-sanitize-recover=all"]


def run(tmp_path, places):
    exe = str(tmp_path / "driver")
    r = subprocess.run(["g++"] + FLAGS + ["-I", places, os.path.join(ROOT, "tests", "sanitize", "balance_places_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return subprocess.run([exe, "60"], capture_output=True, text=True)


CSRC = os.path.join(ROOT, "quantized_moe_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_sum_is_found(tmp_path):
    r = run(tmp_path, CSRC)
    assert r.returncode == 0 and r.stdout == "OK\n", (r.stdout[-2000:], r.stderr[-2000:])


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
@pytest.mark.parametrize("right,wrong,message", [
    ("T > 0 ? (T + 8191) / 8192 : 1", "(T + 8191) / 8192", "division by zero"),   # a call without tokens
    ("first < end && first < block", "first < block", "a place without a sum"),   # an empty sequence at the last token
    ("at + run > first && at < end", "at + run > first", "a place without a sum"),
    ("at > first ? at : first", "at", "a place without a sum"),
])
def test_the_check_sees_wrong_places(tmp_path, right, wrong, message):
    """Mistakes planted into a copy of the functions."""
    text = open(os.path.join(CSRC, "balance_places.hpp")).read()
    assert text.count(right) == 1
    (tmp_path / "balance_places.hpp").write_text(text.replace(right, wrong))
    r = run(tmp_path, str(tmp_path))
    assert r.returncode != 0 and message in r.stdout + r.stderr
