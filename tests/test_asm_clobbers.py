"""Inline assembly of the kernels, read as text: a statement that sets a register by name tells the compiler so."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_quantized_mat_quantize_amd", "csrc")


def statements(text):
    """The text of each asm statement, from its opening parenthesis to the one that closes it, strings passed over."""
    for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", text):
        depth, i = 1, m.end()
        while depth:
            if text[i] == '"':
                i += 1
                while text[i] != '"':
                    i += 2 if text[i] == "\\" else 1
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield text[m.end():i - 1], text.count("\n", 0, m.start()) + 1


def sets_m0(statement):
    return re.search(r"\bs_\w+\s+m0\s*,", statement) is not None


def test_m0_is_named():
    """m0 holds where a direct load puts its data; the compiler may keep a value of its own in it."""
    found, unnamed = 0, []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h"))):
        with open(path) as f:
            for statement, line in statements(f.read()):
                if sets_m0(statement):
                    found += 1
                    if '"m0"' not in statement:
                        unnamed.append(f"{os.path.basename(path)}:{line}")
    assert found and not unnamed, unnamed


def test_the_reader_of_statements():
    text = 'int a;\nasm volatile("s_mov_b32 m0, %0\\n\\t(x \\" " ::"s"(f(1)) : "memory");\nasm("v_mov_b32 %0, 0" : "=v"(b));'
    got = list(statements(text))
    assert [line for _, line in got] == [2, 3]
    assert [sets_m0(s) for s, _ in got] == [True, False]
    assert got[0][0].endswith(': "memory"')
