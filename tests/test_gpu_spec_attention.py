"""The decoding example behind a shared prompt: every layer's attention, of
every request and step, against the plain 64-bit implementation over the pages
that the step left in the cache, within its bound (tests/kv4_ref.py)."""
import numpy as np
import pytest

import kv4_ref as R
from gpu_util import say

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_quantized_decode_pn3t_amd import spec_step as S  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield


@pytest.mark.parametrize("dim,q_heads,heads,page,sandwich", [(64, 8, 2, 16, True), (128, 6, 1, 16, False),
                                                             (256, 12, 2, 32, False)])
def test_every_request(monkeypatch, dim, q_heads, heads, page, sandwich):
    say("spec_step attention dim=%d heads=%d/%d page=%d" % (dim, q_heads, heads, page))
    model = S.Decoder(2, 512, q_heads, heads, dim, 640, seed=dim, sandwich=sandwich)
    req = S.Requests(model, 4, 300, page)
    real, seen = S.Requests._attend, []

    def attend(self, cache, q16, out, T, max_q):
        real(self, cache, q16, out, T, max_q)
        torch.cuda.synchronize()
        pages = cache.keep.view(cache.desc.num_pages, -1).cpu().numpy()
        q_start, kv = self.q_start.cpu().numpy(), self.kv_len.cpu().numpy()
        want, bound = R.attend(q16.cpu().numpy().reshape(T, q_heads, dim).astype(np.float64), pages, page, heads, dim, q_start,
                               kv, self.table.cpu().numpy(), np.float64(np.float32(dim ** -0.5)), 0, 0, len(pages))
        got = out.cpu().numpy().reshape(want.shape).astype(np.float64)
        assert (np.abs(got - want) <= bound).all(), (len(seen), np.argwhere(~(np.abs(got - want) <= bound))[:3].tolist())
        seen.append((self.prefix is not None, np.diff(q_start).tolist()))
    monkeypatch.setattr(S.Requests, "_attend", attend)
    g = np.random.default_rng(dim)

    def some(k):
        return torch.from_numpy(g.integers(0, 640, k, dtype=np.int32)).cuda()

    def u(k):
        return torch.from_numpy(g.random((4, k), dtype=np.float32)).cuda()
    assert req.share(some(150)) == 150 // page * page
    lengths = [1, 30, 7, 17]
    req.prompt(some(sum(lengths)), lengths, u(1))
    for k in (0, 3, 0):
        req.step(u(k + 1), some(4 * k).reshape(4, k) if k else None)
    req.check()
    layers = len(model.layers)
    assert [x for x, _ in seen] == [False] * layers + [True] * 4 * layers
    assert seen[layers][1] == lengths and seen[-1][1] == [1] * 4
