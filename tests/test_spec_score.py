"""The decoding example's scores on the CPU: what is refused before any call."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from bit_quantized_decode_pn3t_amd import spec_step as S  # noqa: E402


def requests(monkeypatch):
    model = SimpleNamespace(device=torch.device("cpu"), heads=1, dim=64, layers=[0], window=0, vocab=100)
    calls = []
    monkeypatch.setattr(S.B, "pn_logprobs", lambda *a, **kw: calls.append(a))
    return S.Requests(model, 3, 100, 16), calls


@pytest.mark.parametrize("logits,tokens", [
    (torch.zeros(3, 100, dtype=torch.bfloat16), torch.zeros(3, 1)), (torch.zeros(3, 100, dtype=torch.float64), torch.zeros(3, 1)),
    (torch.zeros(2, 100), torch.zeros(3, 1)), (torch.zeros(3, 99), torch.zeros(3, 1)), (torch.zeros(300), torch.zeros(3, 1)),
])
def test_logits_that_are_not_rows_of_the_vocabulary(monkeypatch, logits, tokens):
    req, calls = requests(monkeypatch)
    with pytest.raises(ValueError):
        req.score(logits, tokens)
    assert calls == []


@pytest.mark.parametrize("kind,name", [(torch.float32, "f32"), (torch.float16, "f16")])
def test_types_and_strides(monkeypatch, kind, name):
    req, calls = requests(monkeypatch)
    wide = torch.arange(3 * 128).reshape(3, 128).to(kind)
    req.score(wide[:, :100], torch.zeros(3, 2), top=4)
    req.score(wide[:, :100].t().contiguous().t(), torch.zeros(3, 2))
    req.score(wide[:1, :100].expand(3, 100), torch.zeros(3, 2))
    assert [a[1:5] for a in calls] == [(name, 128, 3, 100), (name, 100, 3, 100), (name, 100, 3, 100)]
    assert torch.equal(calls[1][0], wide[:, :100]) and calls[1][0].stride() == (100, 1)


def test_tokens_past_32_bits_are_outside_of_the_vocabulary(monkeypatch):
    req, calls = requests(monkeypatch)
    req.score(torch.zeros(3, 100), torch.tensor([[5, 2 ** 32 + 5], [-1, 99], [100, -2 ** 40]]))
    assert calls[0][6].tolist() == [[5, -1], [-1, 99], [-1, -1]]
