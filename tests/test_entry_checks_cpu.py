"""Checks around the C entries and in the binding that need no GPU."""
import shutil
import subprocess

import pytest
import torch

import gated_deltanet_linear_11_gb300 as gdn
from gated_deltanet_linear_11_gb300 import build


@pytest.mark.skipif(shutil.which("nm") is None, reason="needs nm")
def test_no_allocation_that_throws():
    """An exception must not leave a C entry: the library allocates nothing on the host by the
    throwing operator new, and has no container that can exceed its length."""
    out = subprocess.run(["nm", "-u", build.build()], capture_output=True, text=True, check=True)
    names = {line.split()[-1].split("@")[0] for line in out.stdout.splitlines() if line.split()}
    assert not names & {"_Znwm", "_Znam", "_ZSt17__throw_bad_allocv",
                        "_ZSt20__throw_length_errorPKc", "__cxa_throw"}


class _OnDevice(torch.Tensor):
    """A host tensor that says it lives on a GPU."""
    is_cuda = True


def test_too_few_device_offsets_are_refused():
    """The kernels index the device offsets by the host copy's count."""
    host = torch.tensor([0, 3, 5, 9], dtype=torch.int32)
    for n in (1, 3):
        short = host[:n].clone().as_subclass(_OnDevice)
        for pair in (gdn._offsets, gdn._seqlens):
            with pytest.raises(ValueError, match="%d entries and cu_seqlens_host 4" % n):
                pair(short, host)
    for more in (0, 2):                # a longer device tensor does no harm
        dev = torch.cat((host, host[:more])).as_subclass(_OnDevice)
        assert gdn._offsets(dev, host)[0] is dev and gdn._offsets(dev, host)[1] is host


def on(device):
    class Fake(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return device
    return torch.zeros(2).as_subclass(Fake)


def test_entries_run_on_the_device_of_their_tensors(monkeypatch):
    """The C side launches on the current device: a call whose tensors live on another one makes
    that current for as long as it runs."""
    now = [0]

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.was, now[0] = now[0], self.d

        def __exit__(self, *exc):
            now[0] = self.was
    monkeypatch.setattr(gdn, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)

    @gdn._on_device
    def entry(q, fail=False):
        if fail:
            raise ValueError
        return now[0]
    assert entry(on(0)) == 0 and entry(on(1)) == 1 and entry(q=on(2)) == 2 and now[0] == 0
    with pytest.raises(ValueError):
        entry(on(1), fail=True)
    assert now[0] == 0
    launching = [n for n in gdn.__all__ if n.startswith("gdn_") and not n.endswith(
        ("_size", "_hint", "gdn_kv_cache"))]
    assert len(launching) == 14
    for name in launching:
        assert hasattr(getattr(gdn, name), "__wrapped__"), name


def test_tensors_of_different_devices_are_refused():
    gdn._need_cuda(on(1), None, on(1))
    with pytest.raises(ValueError, match="different devices"):
        gdn._need_cuda(on(1), None, on(0))
    with pytest.raises(ValueError, match="CUDA device"):
        gdn._need_cuda(on(0), torch.zeros(1))
    with pytest.raises(ValueError, match="CUDA device"):
        gdn._need_cuda(torch.zeros(1), None)
