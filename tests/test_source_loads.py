"""Kernels that start over their predecessor's tail read nothing through the read-only path, whose data nobody may write while
the kernel lives: no __ldg, and no `const T *__restrict__` that the compiler would turn into one (host only, by the text)."""
import re
from pathlib import Path

CSRC = Path(__file__).resolve().parents[1] / "param_buffers_gb300" / "csrc"


def code(path):
    text = re.sub(r"/\*.*?\*/", "", path.read_text(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def test_no_read_only_loads():
    files = sorted(p for p in CSRC.iterdir() if p.suffix in (".cu", ".cuh"))
    assert len(files) > 10
    found = [(p.name, m.group(0)) for p in files for m in
             re.finditer(r"__ldg\s*\(|const\s+\w+\s*\*\s*__restrict__|ld\.global\.nc", code(p))]
    assert not found, found
