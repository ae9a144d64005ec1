"""The decoding example's shared prompt on the CPU: what is entered, and what is refused."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from bit_quantized_decode_pn3t_amd import spec_step as S  # noqa: E402


def requests(monkeypatch, window=0):
    model = SimpleNamespace(device=torch.device("cpu"), heads=1, dim=64, layers=[0], window=window)
    req = S.Requests(model, 3, 100, 16)
    ran = []

    def forward(self, tokens, new_len, max_q):
        ran.append((tokens.tolist(), new_len.tolist(), max_q))
        self.table[0, :2] = torch.tensor([7, 5], dtype=torch.int32)
    monkeypatch.setattr(S.Requests, "_forward", forward)
    return req, ran


def test_whole_pages_are_entered_once(monkeypatch):
    req, ran = requests(monkeypatch)
    assert req.share(torch.arange(15)) == 0 and ran == [] and req.prefix is None
    assert req.share(torch.arange(45)) == 32
    assert ran == [(list(range(32)), [32, 0, 0], 32)]
    assert req.table[:, :2].tolist() == [[7, 5]] * 3 and req.prefix.tolist() == [[7, 5]]
    assert req.ctx.tolist() == [32] * 3 and req.held.tolist() == [2] * 3 and req.longest == 32
    assert req.g_start.tolist() == [0, 3] and req.shared.tolist() == [2]


def test_refusals(monkeypatch):
    req, ran = requests(monkeypatch)
    with pytest.raises(ValueError):
        req.share(torch.arange(130))  # 8 whole pages, 128 tokens, past max_len = 112
    req.longest = 1
    with pytest.raises(ValueError):
        req.share(torch.arange(45))  # not first
    req, ran = requests(monkeypatch)
    req.share(torch.arange(45))
    with pytest.raises(ValueError):
        req.share(torch.arange(45))  # a second one
    req, ran = requests(monkeypatch, window=8)
    with pytest.raises(ValueError):
        req.share(torch.arange(45))
    assert ran == []
