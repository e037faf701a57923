"""What the compiler cannot check about the kernels' sources."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_moe_amd", "csrc")


def asm_statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[i], 0)
                i += 1
            yield os.path.basename(path), text[m.end(): i - 1]


def test_asm_that_writes_m0_says_so():
    """m0 is a register that the compiler may keep a value in: a statement that writes it has to name it."""
    writers = [(name, s) for name, s in asm_statements() if re.search(r"\bs_mov_b32\s+m0\b", s)]
    assert writers
    for name, s in writers:
        assert '"m0"' in s.split("::")[-1], (name, s)
