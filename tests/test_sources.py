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


def operands(statement):
    """(instructions, [(constraint, is an output)]) of an asm statement."""
    strings = re.compile(r'"((?:[^"\\]|\\.)*)"')
    template, at = "", 0
    while True:  # the literals (and macro arguments) before the first colon outside of one
        m, colon = strings.search(statement, at), statement.find(":", at)
        if m is None or (0 <= colon < m.start()):
            break
        template += m.group(1)
        at = m.end()
    rest = statement[at:]
    found = re.findall(r'"([^"]*)"\s*\(', rest)
    instructions = [i for i in re.split(r"\\n\\t|\\n|\\t", template) if i.strip()]
    return instructions, found


def test_asm_outputs_written_before_an_input_is_read_have_registers_of_their_own():
    """Without '&' the compiler may give such an output the register of an input that is still needed."""
    seen = 0
    for name, s in asm_statements():
        instructions, constraints = operands(s)
        uses = [re.findall(r"%(\d+)", i) for i in instructions]
        inputs = [i for i, c in enumerate(constraints) if c[:1] not in "=+" and "v" in c]
        for o, c in enumerate(constraints):
            if c[:1] not in "=+" or "v" not in c:
                continue
            writes = [n for n, u in enumerate(uses) if u and int(u[0]) == o]
            reads = [n for n, u in enumerate(uses) if any(int(x) in inputs for x in u[1:])]
            seen += 1
            if writes and reads and writes[0] < reads[-1]:
                assert "&" in c, (name, o, instructions)
    assert seen > 10
