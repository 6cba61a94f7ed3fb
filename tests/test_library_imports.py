"""The library allocates no memory, on the host either: it imports no allocator."""
import shutil
import subprocess

import pytest

from gated_deltanet_recurrence_gdn_amd import binding as gb


def test_no_allocator_is_imported():
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("nm is not available")
    names = subprocess.run([nm, "-D", "-C", "--undefined-only", gb.library_path()], check=True, capture_output=True, text=True).stdout
    assert "hipLaunchKernel" in names
    bad = [n for n in names.split("\n") if any(w in n for w in ("operator new", "malloc", "calloc", "hipMalloc", "hipHostMalloc"))]
    assert not bad, bad
