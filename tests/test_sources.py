"""Every header of the repository is included by a source beside it or above it:
no copy lies about that nothing reaches."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OTHER = {".git", "_work", "gpurun_out", "_build", "__pycache__", ".pytest_cache"}


def files(*ends):
    for at, dirs, names in os.walk(ROOT):
        dirs[:] = [d for d in dirs if d not in OTHER]
        for n in names:
            if n.endswith(ends):
                yield os.path.join(at, n)


def test_every_header_is_included():
    included = set()
    for path in files(".hip", ".h", ".c", ".cpp"):
        with open(path) as f:
            for name in re.findall(r'^\s*#include\s+"([^"]+)"', f.read(), re.M):
                included.add(os.path.normpath(os.path.join(os.path.dirname(path), name)))
    left = [os.path.relpath(h, ROOT) for h in files(".h") if h not in included]
    assert not left, left
