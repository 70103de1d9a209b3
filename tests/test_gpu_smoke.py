"""smoke() reaches every entry that launches kernels of its own."""
import pytest
import torch

import __graft_entry__ as entry

pytestmark = pytest.mark.gpu

gdn = pytest.importorskip("gated_deltanet_linear_11_gb300")


def test_smoke_calls_every_operator(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    called = set()
    lib = gdn.load()

    class Spy:
        def __getattr__(self, name):
            called.add(name)
            return getattr(lib, name)
    monkeypatch.setattr(gdn._lib, "load", lambda *a: Spy())
    entry.smoke()
    assert called >= {"gdn_layer_prefill", "gdn_recurrent_decode", "gdn_linear_prefill",
                      "gdn_linear_decode", "gdn_kv_append", "gdn_kv_read", "gdn_kv_attention"}
