"""Properties of the kernel sources that no run can show reliably."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "chunked_linear_recurrence_gated_gb300", "csrc")


def asm_statements():
    """(file, line, text) of every inline-assembly statement of the kernels."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            text = f.read()
        for m in re.finditer(r"\basm\b\s*(volatile)?\s*\(", text):
            depth, i, quoted = 1, m.end(), False
            while depth:
                c = text[i]
                if c == '"' and text[i - 1] != "\\":
                    quoted = not quoted
                elif not quoted:
                    depth += (c == "(") - (c == ")")
                i += 1
            yield os.path.basename(path), text.count("\n", 0, m.start()) + 1, text[m.start():i]


def test_asynchronous_copies_are_compiler_barriers():
    """A thread's private slots of shared memory are filled by cp.async and read with
    ordinary loads, with no block barrier in between: the copies and their waits
    themselves have to keep the compiler from moving those loads across them."""
    found = [s for s in asm_statements() if "cp.async" in s[2]]
    assert len(found) >= 8
    bad = [(f, line) for f, line, text in found if '"memory"' not in text or "volatile" not in text]
    assert not bad, bad


def test_flags_between_warps_are_fenced():
    """A thread that tells others through a plain flag in shared memory what it has seen of the
    teams' events fences in between, and so does who acts on the flag: the event itself orders
    the teams' accesses for the thread that waited for it only."""
    with open(os.path.join(CSRC, "gdn_lin_tc.cu")) as f:
        text = f.read()
    tells = re.findall(r"auto see = .*?\n      };", text, re.S)
    assert len(tells) == 2
    for body in tells:
        assert "__threadfence_block();" in body.split("seen[tell]")[0], body
    waits = [m.end() for m in re.finditer(r"while \(!\*abort && [^{]*seen\[", text)]
    assert len(waits) == 2
    for at in waits:
        behind = text[at:at + 700]
        assert "__threadfence_block();" in behind.split("load(")[0], behind
