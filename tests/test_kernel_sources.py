"""Checks of the kernels' sources that need no GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "replicated_fp8_sparse_amd", "csrc")


def asm_statements(text):
    """Every asm statement: (template, [outputs, inputs, clobbers] as text)."""
    for at in re.finditer(r"\basm\s*(?:volatile\s*)?\(", text):
        depth, i, quoted, cuts = 1, at.end(), False, [at.end()]
        while depth:
            c = text[i]
            if quoted:
                i += c == "\\"
                quoted = c != '"'
            elif c == '"':
                quoted = True
            elif c == "(":
                depth += 1
            elif c == ")":
                depth -= 1
            elif c == ":" and depth == 1:
                cuts.append(i + 1)
            i += 1
        cuts.append(i)
        parts = [text[a:z - 1] for a, z in zip(cuts, cuts[1:])]
        yield parts[0], (parts[1:] + ["", "", ""])[:3]


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith(".hip")))
def test_asm_declares_m0_where_it_writes_it(name):
    with open(os.path.join(CSRC, name)) as f:
        for template, (_, _, clobbers) in asm_statements(f.read()):
            if re.search(r"\bs_\w+\s+m0\b", template):
                assert '"m0"' in clobbers, template


def test_statements_are_found():
    got = list(asm_statements('asm("" : "+s"(r)); asm volatile("s_mov_b32 m0, %0\\n\\tx" ::"s"(f(a)), "v"(b) : "memory", "m0");'))
    assert len(got) == 2 and got[1][1][2].strip() == '"memory", "m0"' and got[0][1][0].strip() == '"+s"(r)'
