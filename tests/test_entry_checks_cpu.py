"""Checks around the C entries and in the binding that need no GPU."""
import shutil
import subprocess

import pytest

from gated_deltanet_linear_11_gb300 import build


@pytest.mark.skipif(shutil.which("nm") is None, reason="needs nm")
def test_no_allocation_that_throws():
    """An exception must not leave a C entry: the library allocates nothing on the host by the
    throwing operator new, and has no container that can exceed its length."""
    out = subprocess.run(["nm", "-u", build.build()], capture_output=True, text=True, check=True)
    names = {line.split()[-1].split("@")[0] for line in out.stdout.splitlines() if line.split()}
    assert not names & {"_Znwm", "_Znam", "_ZSt17__throw_bad_allocv",
                        "_ZSt20__throw_length_errorPKc", "__cxa_throw"}
