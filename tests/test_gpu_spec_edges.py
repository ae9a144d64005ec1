"""The decoding example on the GPU where its cache ends: requests that reach
max_len, and a shortage of pages."""
import numpy as np
import pytest

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


def start(max_len, lengths, seed):
    model = S.Decoder(1, 256, 2, 1, 64, 320, seed=seed)
    g = np.random.default_rng(seed)
    req = S.Requests(model, len(lengths), max_len, 16)
    prompt = torch.from_numpy(g.integers(0, 320, sum(lengths), dtype=np.int32)).cuda()
    return g, req, prompt


def pages_of(req):
    table, held = req.table.cpu().numpy(), req.held.cpu().numpy()
    return [[int(p) for p in table[i, :held[i]]] for i in range(req.batch)]


def step(g, req, k):
    u = torch.from_numpy(g.random((req.batch, k + 1), dtype=np.float32)).cuda()
    drafts = torch.from_numpy(g.integers(0, 320, (req.batch, k), dtype=np.int32)).cuda()
    return req.step(u, drafts, greedy=True)


def test_until_full():
    """Steps up to max_len and not past it: every page belongs to one request, no token is lost."""
    g, req, prompt = start(64, [10, 40, 33], 1)
    req.prompt(prompt, [10, 40, 33], torch.zeros((3, 1), device="cuda"), greedy=True)
    steps = 0
    with pytest.raises(ValueError):
        while steps < 64:
            step(g, req, 5)
            steps += 1
    say("full after %d steps, %s" % (steps, req.ctx.tolist()))
    assert 64 - 6 < int(req.ctx.max()) <= 64 and int(req.held.max()) <= 4
    req.check()
    pages = sum(pages_of(req), [])
    assert len(set(pages)) == len(pages) and min(pages) >= 0 and max(pages) < 12
    for _ in range(64 - int(req.ctx.max())):
        step(g, req, 0)
    assert int(req.ctx.max()) == 64
    req.check()


def test_shortage():
    """Fewer pages than the requests need: the tokens that find no place are
    reported, and no page goes to two requests."""
    g, req, prompt = start(160, [20, 37, 33], 2)
    req.free[9:] = -1
    req.prompt(prompt, [20, 37, 33], torch.zeros((3, 1), device="cuda"), greedy=True)
    req.check()  # 2 + 3 + 3 pages
    for _ in range(24):  # each brings every request a token at least, which takes more than nine pages
        step(g, req, 3)
    with pytest.raises(RuntimeError):
        req.check()
    pages = [p for p in sum(pages_of(req), []) if p >= 0]
    assert len(set(pages)) == len(pages) == 9
