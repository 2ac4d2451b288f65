"""Inline assembly of the kernels' sources: what a block writes by name it says."""
import glob
import os
import re

from zero_partitioned_optimizer_flatten_amd import build as zb


def blocks():
    """(file, text, clobbers) of every asm statement."""
    for path in sorted(glob.glob(os.path.join(zb.CSRC, "*.h*"))):
        source = open(path).read()
        for m in re.finditer(r"\basm\s+volatile\s*\(", source):
            depth, at, quoted = 1, m.end(), False
            while depth:
                c = source[at]
                if c == '"':
                    quoted = not quoted
                elif not quoted:
                    depth += (c == "(") - (c == ")")
                at += 1
            body = source[m.end():at - 1]
            parts = [""]
            for piece in re.split(r'("[^"]*")', body):
                if piece.startswith('"'):
                    parts[-1] += piece
                else:
                    first, *more = piece.split(":")
                    parts[-1] += first
                    parts += more
            text = "".join(re.findall(r'"([^"]*)"', parts[0])).replace("\\n", "\n").replace("\\t", " ")
            yield os.path.basename(path), text, re.findall(r'"([^"]*)"', parts[3]) if len(parts) > 3 else []


def test_named_registers_are_clobbers():
    seen = 0
    for name, text, clobbers in blocks():
        for line in text.splitlines():
            m = re.match(r"\s*\w+\s+(m0|vcc|exec|scc|[sv]\d+|[sv]\[\d+:\d+\])\s*,", line)
            if m:
                seen += 1
                assert m.group(1) in clobbers, (name, line, clobbers)
    assert seen >= 1


def test_loads_to_lds_and_barriers_are_not_moved_past():
    """Blocks that touch memory or other waves hold the compiler's own accesses in place."""
    seen = 0
    for name, text, clobbers in blocks():
        if re.search(r"\b(buffer_load|global_load|s_barrier|s_waitcnt)", text):
            seen += 1
            assert "memory" in clobbers, (name, text, clobbers)
    assert seen >= 6
