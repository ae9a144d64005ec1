"""The decoding example with a shared prompt, sandwich blocks and scores: plan,
store, both kinds of attention, the norms between blocks, verification and log
probabilities together.

A shared prompt changes which kernels read the cache, not what is in it: greedy
tokens are those of prompts entered whole, up to the first whose two best
logits are closer than 0.02 of the logits' deviation (rounding of fp16 hidden
states, 2^-11 a value, is far below that).  The same holds for the norms
between blocks, against torch's."""
import numpy as np
import pytest

import step_ref as R
from gpu_util import say

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_quantized_decode_pn3t_amd import _binding as B  # noqa: E402
from bit_quantized_decode_pn3t_amd import spec_step as S  # noqa: E402

CLOSE = 0.02
STEPS = 12


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield


def tokens_of(req, first, logits, steps):
    """Greedy tokens [B, steps + 1], and where they are certain."""
    got, sure = [first], []
    for i in range(steps + 1):
        top = logits.topk(2, 1).values
        sure.append(top[:, 0] - top[:, 1] > CLOSE * logits.std(1))
        if i == steps:
            break
        out, _, logits = req.step(torch.zeros((req.batch, 1), device="cuda"), greedy=True)
        got.append(out[:, 0])
    req.check()
    return torch.stack(got, 1).cpu().numpy(), torch.stack(sure, 1).cpu().numpy()


def agree(a, b, sure):
    same = 0
    for x, y, s in zip(a, b, sure):
        n = len(x) if s.all() else int(np.argmin(s))
        assert x[:n].tolist() == y[:n].tolist()
        same += n
    assert same >= 6  # and something was compared


@pytest.mark.parametrize("dim,q_heads,heads,page,sandwich", [(64, 8, 2, 16, False), (128, 6, 1, 16, True),
                                                             (256, 12, 2, 32, False), (128, 12, 2, 64, False)])
def test_shared_prompt_as_whole_prompts(dim, q_heads, heads, page, sandwich):
    say("spec_step shared dim=%d heads=%d/%d page=%d sandwich=%d" % (dim, q_heads, heads, page, sandwich))
    model = S.Decoder(2, 512, q_heads, heads, dim, 640, seed=dim, sandwich=sandwich)
    g = np.random.default_rng(dim)
    common = torch.from_numpy(g.integers(0, 640, 333, dtype=np.int32)).cuda()
    lengths = [1, 5, 40, 17]
    own = torch.from_numpy(g.integers(0, 640, sum(lengths), dtype=np.int32)).cuda()
    u = torch.zeros((4, 1), device="cuda")
    whole = S.Requests(model, 4, 420, page)
    parts, at = [], 0
    for n in lengths:
        parts += [common, own[at:at + n]]
        at += n
    out, _, logits = whole.prompt(torch.cat(parts), [333 + n for n in lengths], u, greedy=True)
    want, sure = tokens_of(whole, out[:, 0], logits, STEPS)

    req = S.Requests(model, 4, 420, page)
    count = req.share(common)
    assert count == 333 // page * page
    rest, at, parts = common[count:], 0, []
    for n in lengths:
        parts += [rest, own[at:at + n]]
        at += n
    out, _, logits = req.prompt(torch.cat(parts), [333 - count + n for n in lengths], u, greedy=True)
    assert B.pn_variant_name(B.pn_last_variant()) == "spec_verify"
    got, _ = tokens_of(req, out[:, 0], logits, STEPS)
    agree(got, want, sure)
    # one copy of the shared pages, and the same lengths
    assert (req.table[:, :count // page] == req.table[:1, :count // page]).all()
    assert req.ctx.tolist() == whole.ctx.tolist() == [333 + n + STEPS for n in lengths]
    used = req.table[:, :].unique()
    assert used[used >= 0].numel() < whole.table[whole.table >= 0].numel()


def test_sandwich_as_plain_torch(monkeypatch):
    model = S.Decoder(3, 512, 8, 2, 64, 640, seed=3, sandwich=True)
    g = np.random.default_rng(3)
    prompt = torch.from_numpy(g.integers(0, 640, 60, dtype=np.int32)).cuda()

    def run():
        req = S.Requests(model, 2, 100, 16)
        out, _, logits = req.prompt(prompt, [25, 35], torch.zeros((2, 1), device="cuda"), greedy=True)
        return tokens_of(req, out[:, 0], logits, STEPS)
    want, sure = run()
    calls = []

    def plain(self, h, y, z, w, x):
        calls.append(y is None)
        if y is not None:
            h.add_(self.model.mix * torch.sigmoid(z) * S.norm(y) * w["post"])
        x.copy_(S.norm(h).half())
    monkeypatch.setattr(S.Requests, "_between", plain)
    got, _ = run()
    agree(got, want, sure)
    assert calls.count(True) == STEPS + 1 and calls.count(False) == 3 * (STEPS + 1)


def test_scores_of_a_step():
    model = S.Decoder(1, 512, 8, 2, 64, 1111, seed=9)
    req = S.Requests(model, 3, 64, 16)
    g = np.random.default_rng(9)
    u = torch.from_numpy(g.random((3, 1), dtype=np.float32)).cuda()
    req.prompt(torch.from_numpy(g.integers(0, 1111, 9, dtype=np.int32)).cuda(), [2, 3, 4], u)
    drafts = torch.from_numpy(g.integers(0, 1111, (3, 2), dtype=np.int32)).cuda()
    u = torch.from_numpy(g.random((3, 3), dtype=np.float32)).cuda()
    out, accepted, logits = req.step(u, drafts)
    logp, entropy, ids, best = req.score(logits, out.reshape(-1, 1), top=4, scale=0.5)
    want, H, w_ids, w_best, d, d_h = R.logprobs(logits.cpu().numpy(), 0.5, out.reshape(-1, 1).cpu().numpy(), 4)
    assert np.array_equal(ids.cpu().numpy(), w_ids)
    with np.errstate(invalid="ignore"):
        for got, ref, bound in ((logp, want, d[:, None]), (entropy, H, d_h), (best, w_best, d[:, None])):
            got = got.cpu().numpy()
            assert ((got == ref) | (np.abs(got - ref) <= bound + R.U * np.abs(ref))).all()
    given = out.reshape(-1).cpu().numpy() >= 0
    assert np.isfinite(logp.cpu().numpy()[given]).all() and np.isneginf(logp.cpu().numpy()[~given]).all()
