"""Inline assembly in the kernels leaves the wavefront's state as it was or says what it changes: M0 is put
back or named as clobbered, SCC named, and the lanes that were active are saved before EXEC is narrowed
and put back behind (CPU only, the sources)."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "quantized_moe_sigmoid_amd", "csrc", "*.h*")))


def _statements(src):
    """(code, everything behind it) of each asm statement with a body."""
    for m in re.finditer(r"\basm\s+volatile\s*\(", src):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(src[i], 0)
            i += 1
        body = src[m.end():i - 1]
        code = re.match(r'\s*((?:"(?:[^"\\]|\\.)*"\s*)+)', body).group(1)
        text = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', code)).replace("\\n", "\n").replace("\\t", "")
        yield text, body[len(code):]


def _restored(lines, reg):
    """Does the last instruction that writes reg put back what an instruction before the first such saved?"""
    writes = [n for n, x in enumerate(lines) if len(x) > 1 and re.split(r"[ ,]+", x[1])[0] == reg or "saveexec" in x[0] and reg == "exec"]
    saves = {re.split(r"[ ,]+", x[1])[0]: n for n, x in enumerate(lines)
             if "saveexec" in x[0] and reg == "exec" or x[0].startswith("s_mov_b") and re.split(r"[ ,]+", x[1])[1] == reg}
    source = re.split(r"[ ,]+", lines[writes[-1]][1])[1]
    return lines[writes[-1]][0].startswith("s_mov_b") and source in saves and saves[source] <= writes[0]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_asm_declares_what_it_changes(path):
    for text, rest in _statements(open(path).read()):
        lines = [x.split(None, 1) for x in text.split("\n") if x.strip()]
        written = {re.split(r"[ ,]+", x[1])[0] for x in lines if len(x) > 1 and x[0].startswith("s_")}
        assert not written & {"exec_lo", "exec_hi"}, text
        if "m0" in written:
            assert '"m0"' in rest or _restored(lines, "m0"), text
        if "exec" in written or "saveexec" in text:
            assert _restored(lines, "exec"), text
        if "saveexec" in text:
            assert '"scc"' in rest, text
