"""Building the library (no GPU): the sources compile, and what is built is
what the binding loads."""
from __future__ import annotations

import os
import subprocess
import sys

from l2_row_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_sources_build_and_the_binding_loads():
    """Every source compiles (at once where the library is up to date), and
    every name that the binding declares is in the library."""
    assert build.build() == build.LIB
    code = "from l2_row_b200 import ds; assert all(hasattr(ds.lib(), n) for n in ds.EXPORTS)"
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)
