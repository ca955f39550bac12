"""Sources with matrix instructions have no instructions in inline assembly: the
compiler puts the waits that a matrix instruction's (or an exponential's) result
needs before readers that it knows, and does not look into an asm statement.
Empty ones, which only hold a value in a register, are no instructions."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_dequant_matrix_amd", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h")))


def _asm(text):
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"\basm\b(?:\s+volatile)?\s*\(\s*((?:\"[^\"]*\"\s*)+)", text)


def test_the_search_finds_statements():
    assert _asm('asm("v_nop"); asm volatile("" : "+v"(x)); // asm("no")') == ['"v_nop"', '"" ']


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_instructions_in_asm_beside_matrix_instructions(path):
    text = open(path).read()
    # step_device.h's helpers stand beside the matrix instructions of the files that include it
    if "__builtin_amdgcn_mfma" in text or path.endswith(".h"):
        assert all(not s.replace('"', "").strip() for s in _asm(text)), path
