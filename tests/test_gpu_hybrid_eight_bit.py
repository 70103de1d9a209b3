"""The example stack with 8-bit projections: norms, 8-bit rows and products together."""
import pytest
import torch

from test_gpu_hybrid import _cu, _example

pytestmark = pytest.mark.gpu

KINDS = ("delta", "linear", "delta", "attention")


def _rows(lens, steps):
    gen = torch.Generator().manual_seed(3)
    return [torch.randint(0, 1000, (n + steps,), generator=gen) for n in lens]


def _rel(got, want):
    return float(((got.double() - want.double()).norm(dim=-1) / want.double().norm(dim=-1)).max())


@pytest.mark.parametrize("gate", [False, True])
def test_eight_bit_near_bf16(gate):
    """Codes are off by a step over sqrt(12), 1/440 of a row's largest element, which for rows
    of 512 and 1024 elements is about 4 to 5 times their root mean square: 1.1% of a product
    from either factor, 1.6% together.  Nine products, added up and doubled by the mixers on
    the way, stay under 0.2 of the logits' norm; logits that have nothing in common differ by
    1.4."""
    ex, lens = _example(), [1, 150, 77]
    tokens = torch.cat([r[:n] for r, n in zip(_rows(lens, 1), lens)]).cuda()
    a = ex.HybridStack(KINDS, sequences=3, max_len=256, gate=gate)
    b = ex.HybridStack(KINDS, sequences=3, max_len=256, gate=gate, eight_bit=True)
    assert _rel(b.prefill(tokens, _cu(lens)), a.prefill(tokens, _cu(lens))) <= 0.2


@pytest.mark.parametrize("gate", [False, True])
def test_steps_continue_prompts(gate):
    """As the bf16 stack's: both ways round at the same places, about four of 2^-8 a layer, and
    a code next to a border may take its neighbour, a step of 1/127 of the row's largest."""
    ex, lens, steps = _example(), [1, 150, 77], 3
    rows = _rows(lens, steps)
    a = ex.HybridStack(KINDS, sequences=3, max_len=256, gate=gate, eight_bit=True)
    b = ex.HybridStack(KINDS, sequences=3, max_len=256, gate=gate, eight_bit=True)
    got = [a.prefill(torch.cat([r[:n] for r, n in zip(rows, lens)]).cuda(), _cu(lens))]
    for s in range(steps):
        got.append(a.step(torch.stack([r[n + s] for r, n in zip(rows, lens)]).cuda()))
    for s in range(steps + 1):
        full = [n + s for n in lens]
        want = b.prefill(torch.cat([r[:n] for r, n in zip(rows, full)]).cuda(), _cu(full))
        assert _rel(got[s], want) <= 0.2, s


def test_example_runs(monkeypatch, capsys):
    ex = _example()
    monkeypatch.setattr("sys.argv", ["hybrid_decode.py", "--length", "200", "--tokens", "4",
                                     "--gate", "--eight-bit"])
    ex.main()
    assert "first answer:" in capsys.readouterr().out
