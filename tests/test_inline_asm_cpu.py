"""Inline assembly tells the compiler which registers it writes."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_named_registers_that_are_written_are_clobbers():
    found = 0
    for path in glob.glob(os.path.join(ROOT, "exact_bpe_tokenization_amd", "csrc", "*")):
        if not path.endswith((".h", ".hip")):
            continue
        with open(path) as f:
            text = f.read()
        for statement in re.findall(r"\basm(?:\s+volatile)?\s*\((.*?)\);", text, re.S):
            strings = re.findall(r'"((?:[^"\\]|\\.)*)"', statement)
            code = "\n".join(s for s in strings).replace("\\n", "\n").replace("\\t", "\t")
            for register in set(re.findall(r"^\s*[sv]_\w+\s+(m0|vcc|exec|scc|[sv]\d+)\b", code, re.M)):
                found += 1
                clobbers = re.findall(r'"([^"]*)"', statement.rsplit(":", 1)[1])
                assert register in clobbers, (os.path.basename(path), statement)
    assert found
