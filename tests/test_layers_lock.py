"""The layer operators' entry points share each stream's workspaces, so one lock orders their calls
from several host threads: the built library has exactly one such mutex, not one per entry point."""
from __future__ import annotations

import shutil
import subprocess

import pytest


def test_every_layer_entry_point_queues_under_one_lock(sgemm_lib):
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("needs nm")
    names = subprocess.run([nm, "-C", str(sgemm_lib.library_path())], capture_output=True, text=True,
                           check=True).stdout.splitlines()
    if not names:
        pytest.skip("the library was stripped of its local symbols")
    locks = [n for n in names if n.rstrip().lower().endswith("queueing")]
    assert len(locks) == 1, locks
