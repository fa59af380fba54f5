"""Inline assembly in the kernels names every special register it writes: a value that the
compiler keeps in one of them would be lost otherwise.  No GPU needed."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "trellis_coded_weight_amd", "csrc")
SPECIAL = ("m0", "vcc", "exec")


def statements():
    """(file, [template, outputs, inputs, clobbers]) of every asm statement."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        src = open(path).read()
        for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", src):
            parts, depth, quoted, i = [""], 1, False, m.end()
            while depth:
                c = src[i]
                if c == '"':
                    quoted = not quoted
                if not quoted:
                    depth += {"(": 1, ")": -1}.get(c, 0)
                if c == ":" and not quoted and depth == 1:
                    parts.append("")
                elif depth:
                    parts[-1] += c
                i += 1
            yield os.path.basename(path), parts


def test_written_special_registers_are_clobbered():
    found = 0
    for path, parts in statements():
        code = "".join(re.findall(r'"([^"]*)"', parts[0]))
        clobbers = re.findall(r'"([^"]*)"', parts[3]) if len(parts) > 3 else []
        for instruction in code.replace("\\t", " ").split("\\n"):
            _, _, operands = instruction.strip().partition(" ")
            written = operands.split(",")[0].strip()
            for reg in SPECIAL:
                if re.match(reg + r"\b", written):
                    found += 1
                    assert reg in clobbers, (path, instruction)
    assert found >= 1                      # the loads to LDS take their address from m0
