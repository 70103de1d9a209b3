"""The example stack: a prompt and then single tokens give what the longer prompt gives."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                     "hybrid_decode.py")


def _example():
    spec = importlib.util.spec_from_file_location("hybrid_decode", _PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _cu(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).int()


@pytest.mark.parametrize("kinds", [("linear",), ("attention",),
                                   ("delta", "linear", "delta", "attention")])
def test_steps_continue_prompts(kinds):
    """Both ways round to bf16 at the same places (about four of 2^-8 a layer), in another
    order of sums; a stored key or value next to a rounding border may take the neighbouring
    code.  0.1 of the logits' norm bounds both for four layers; a wrong position, state or
    page gives logits that have nothing in common (1.4)."""
    ex = _example()
    lens, steps = [1, 150, 77], 5
    gen = torch.Generator().manual_seed(3)
    rows = [torch.randint(0, 1000, (n + steps,), generator=gen) for n in lens]
    a = ex.HybridStack(kinds, sequences=3, max_len=256)
    b = ex.HybridStack(kinds, sequences=3, max_len=256)
    got = [a.prefill(torch.cat([r[:n] for r, n in zip(rows, lens)]).cuda(), _cu(lens))]
    for s in range(steps):
        got.append(a.step(torch.stack([r[n + s] for r, n in zip(rows, lens)]).cuda()))
    for s in range(steps + 1):
        full = [n + s for n in lens]
        want = b.prefill(torch.cat([r[:n] for r, n in zip(rows, full)]).cuda(), _cu(full)).double()
        err = (got[s].double() - want).norm(dim=-1) / want.norm(dim=-1)
        assert err.max() <= 0.1, (s, err)


def test_example_runs(monkeypatch, capsys):
    ex = _example()
    monkeypatch.setattr("sys.argv", ["hybrid_decode.py", "--length", "200", "--tokens", "4"])
    ex.main()
    assert "first answer:" in capsys.readouterr().out
