"""What gdn_device_status says of the kernels' status bits: each is told of the operator whose
kernel records it.  The header is plain C++, compiled into a program of the test's own."""
import os
import re
import subprocess

import pytest

from gdn_testutil import ROOT

CSRC = os.path.join(ROOT, "linear_attention_recurrence_gb300", "csrc")
PROGRAM = """
#include <cstdlib>
#include <iostream>
#include "gdn_status.h"
int main(int, char** v) { std::cout << gdn::status_message(std::atoi(v[1]), std::atoi(v[2]), std::atoi(v[3])); }
"""


@pytest.fixture(scope="module")
def say(tmp_path_factory):
    d = tmp_path_factory.mktemp("status")
    (d / "say.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-o", str(d / "say"), str(d / "say.cpp")], check=True)
    return lambda *words: subprocess.run([str(d / "say"), *map(str, words)], capture_output=True, text=True, check=True).stdout


def bits():
    text = open(os.path.join(CSRC, "gdn_status.h")).read()
    return {name: int(value) for name, value in re.findall(r"constexpr int (kDevErr\w+) = (\d+);", text)}


OPERATORS = ("gdn_ssm_scan", "gdn_block_norm", "gdn_kv_attention", "gdn_recurrence_chunked_noalloc")


@pytest.mark.parametrize("names,operators,layout", [
    (["kDevErrTimeout"], ["gdn_ssm_scan"], False), (["kDevErrLayout"], ["gdn_ssm_scan"], True),
    (["kDevErrBlockNorm"], ["gdn_block_norm"], False), (["kDevErrKv"], ["gdn_kv_attention"], False),
    (["kDevErrKvLayout"], ["gdn_kv_attention"], True), (["kDevErrKv", "kDevErrLayout"], ["gdn_kv_attention", "gdn_ssm_scan"], True),
    (["kDevErrKvLayout", "kDevErrBlockNorm"], ["gdn_kv_attention", "gdn_block_norm"], True),
])
def test_operators_over_packed_rows(say, names, operators, layout):
    word = sum(bits()[n] for n in names)
    msg = say(0, 0, word)
    assert f"status word {word})" in msg
    assert [o for o in OPERATORS if o in msg] == [o for o in OPERATORS if o in operators]
    assert ("shared memory" in msg) == layout


def test_the_recurrence(say):
    assert not any(o in say(bits()["kDevErrFlagTimeout"], 0, 0) for o in OPERATORS)
    assert "gdn_recurrence_chunked_noalloc" in say(0, 1, 0)
    assert "exchange between CTAs" in say(4, 0, 0) and "tile ring" in say(8, 0, 0)


def test_bits_are_apart_and_the_caches_kernels_record_their_own():
    values = list(bits().values())
    assert len(set(values)) == len(values) and all(v & (v - 1) == 0 for v in values)
    for name in os.listdir(CSRC):
        if name.startswith("gdn_kv"):
            recorded = re.findall(r"kDevErr\w+", open(os.path.join(CSRC, name)).read())
            assert all(r.startswith("kDevErrKv") for r in recorded), (name, recorded)
