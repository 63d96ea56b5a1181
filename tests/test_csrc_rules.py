"""Rules of the kernels' sources that no run shows: what inline assembly
writes has to be declared, or the compiler may keep a value of its own there."""

import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "sparse_communication_distributed_amd", "csrc", "*")))


def asm_statements(text):
    """(template, operands and clobbers) of each asm statement."""
    for m in re.finditer(r"\basm\s+(?:volatile\s*)?\((.*?)\)\s*;", text, flags=re.S):
        body = m.group(1)
        head = re.match(r'\s*((?:"(?:[^"\\]|\\.)*"\s*)+)', body)
        yield head.group(1), body[head.end():]


def test_assembly_declares_the_registers_it_names():
    seen = 0
    for path in SOURCES:
        for template, rest in asm_statements(open(path).read()):
            named = set(re.findall(r"\b(m0|vcc|exec|scc)\b", template.replace("\\n", " ").replace("\\t", " ")))
            clobbers = rest.split(":")[-1] if rest.count(":") >= 3 else ""
            for reg in named:
                seen += 1
                assert f'"{reg}"' in clobbers, f"{os.path.basename(path)}: {reg} is not declared in {template}"
    assert seen >= 1
