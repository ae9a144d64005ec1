"""The decoding example on the GPU: products, plan, store, attention and
verification together.

Greedy speculative decoding must give the tokens of greedy token-by-token
decoding whatever is drafted.  The two run different kernels (products and
attention of 1 and of k + 1 tokens), whose logits differ by rounding: the
fp16 hidden states by 2^-11 a value, and now and then a cached code by one
step of 1/8 of its block's largest value.  Both are far below 0.02 of the
logits' deviation, so tokens are compared up to the first whose two best
logits are closer than that."""
import numpy as np
import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_quantized_decode_pn3t_amd import _binding as B  # noqa: E402
from bit_quantized_decode_pn3t_amd import spec_step as S  # noqa: E402

CLOSE = 0.02
LENGTHS = [1, 37, 130]
STEPS = 24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield


def start(model, prompt, max_len=260, page=16):
    req = S.Requests(model, len(LENGTHS), max_len, page)
    u = torch.zeros((len(LENGTHS), 1), device="cuda")
    out, accepted, logits = req.prompt(prompt, LENGTHS, u, greedy=True)
    assert not accepted.any()
    return req, out[:, 0], logits


def plain(model, prompt):
    """Tokens [B, STEPS + 1] of token-by-token decoding and where they are certain."""
    req, first, logits = start(model, prompt)
    tokens, sure = [first], []
    for _ in range(STEPS + 1):
        top = logits.topk(2, 1).values
        sure.append(top[:, 0] - top[:, 1] > CLOSE * logits.std(1))
        if len(sure) > STEPS:
            break
        out, _, logits = req.step(torch.zeros((len(LENGTHS), 1), device="cuda"), greedy=True)
        tokens.append(out[:, 0])
    torch.cuda.synchronize()
    assert req.ctx.tolist() == [n + STEPS for n in LENGTHS]
    return torch.stack(tokens, 1).cpu().numpy(), torch.stack(sure, 1).cpu().numpy()


@pytest.mark.parametrize("dim,q_heads,heads,window", [(64, 8, 2, 0), (128, 8, 8, 0), (256, 6, 1, 0), (64, 4, 1, 48)])
@pytest.mark.parametrize("k", [1, 4])
def test_greedy_as_token_by_token(dim, q_heads, heads, window, k):
    model = S.Decoder(2, 512, q_heads, heads, dim, 640, window, 4 if window else 0, seed=dim + k)
    g = np.random.default_rng([dim, k])
    prompt = torch.from_numpy(g.integers(0, 640, sum(LENGTHS), dtype=np.int32)).cuda()
    say("spec_step dim=%d heads=%d/%d window=%d k=%d" % (dim, q_heads, heads, window, k))
    want, sure = plain(model, prompt)
    upto = [int(np.argmin(s)) if not s.all() else STEPS + 1 for s in sure]  # tokens that must agree
    say("agree up to %s of %d" % (upto, STEPS + 1))

    req, first, _ = start(model, prompt)
    got = [[int(t)] for t in first]
    worst = 0
    for _ in range(STEPS // 2):
        drafts = np.zeros((len(LENGTHS), k), np.int32)
        for i, seq in enumerate(got):
            for j in range(k):
                at = len(seq) + j
                right = at <= STEPS and g.random() < 0.75
                drafts[i, j] = want[i, at] if right else g.integers(-1, 641)
        u = torch.from_numpy(g.random((len(LENGTHS), k + 1), dtype=np.float32)).cuda()
        out, accepted, _ = req.step(u, torch.from_numpy(drafts).cuda(), greedy=True)
        out, accepted = out.cpu().numpy(), accepted.cpu().numpy()
        for i, seq in enumerate(got):
            a = int(accepted[i])
            assert np.array_equal(out[i, :a], drafts[i, :a]) and (out[i, a + 1:] == -1).all()
            assert 0 <= out[i, a] < 640
            seq.extend(int(t) for t in out[i, :a + 1])
            worst = max(worst, a)
        assert req.ctx.tolist() == [n + len(seq) - 1 for n, seq in zip(LENGTHS, got)]
    assert worst == k  # some step took every draft
    for i, seq in enumerate(got):
        n = min(upto[i], len(seq), STEPS + 1)
        assert seq[:n] == want[i, :n].tolist(), i
    assert sum(min(n, len(s)) for n, s in zip(upto, got)) >= 6  # and something was compared

    # The first layer's cache depends on tokens and positions alone: what the
    # steps left there, over rejected drafts, is what one long prompt leaves.
    tokens, at, lengths = prompt.cpu().numpy(), 0, []
    rows = []
    for n, seq in zip(LENGTHS, got):
        rows.append(np.concatenate([tokens[at:at + n], np.array(seq[:-1], np.int32)]))
        lengths.append(len(rows[-1]))
        at += n
    whole = S.Requests(model, len(LENGTHS), 260, 64)
    whole.prompt(torch.from_numpy(np.concatenate(rows)).cuda(), lengths,
                 torch.zeros((len(LENGTHS), 1), device="cuda"), greedy=True)
    for i, n in enumerate(lengths):
        kv = []
        for r in (req, whole):
            pos = torch.arange(n, device="cuda")
            slots = r.table[i].long()[pos // r.page_size] * r.page_size + pos % r.page_size
            k_, v_ = (torch.empty((n, heads * dim), device="cuda") for _ in range(2))
            B.pn_kv4_load(r.caches[0], slots, n, k_, v_)
            kv.append((k_, v_))
        for a, b in zip(*kv):
            blocks = b.view(n, -1, 64).abs().amax(-1, keepdim=True)
            diff = (a - b).view(n, -1, 64).abs()
            assert (diff <= blocks * 0.13).all()  # one code's step, 1/8, and the scale's own rounding
            assert (diff > blocks * 2.0 ** -9).float().mean() < 0.001  # codes on a tie alone


def test_sampled_steps():
    """Drafts with their probabilities, sampled: lengths and tokens stay in range."""
    model = S.Decoder(2, 512, 8, 2, 128, 640, seed=5)
    g = np.random.default_rng(5)
    prompt = torch.from_numpy(g.integers(0, 640, sum(LENGTHS), dtype=np.int32)).cuda()
    req, first, _ = start(model, prompt)
    rand = torch.Generator(device="cuda")
    rand.manual_seed(5)
    ctx = np.array(LENGTHS)
    taken = 0
    for _ in range(8):
        noise = torch.empty((3, 3, 640), device="cuda").exponential_(generator=rand)
        tokens, draft = model.draft(req.last, 3, noise)
        out, accepted, _ = req.step(torch.rand((3, 4), generator=rand, device="cuda"), tokens, draft)
        out, accepted, tokens = out.cpu().numpy(), accepted.cpu().numpy(), tokens.cpu().numpy()
        ctx += accepted + 1
        taken += accepted.sum()
        assert req.ctx.tolist() == ctx.tolist()
        for i, a in enumerate(accepted):
            assert np.array_equal(out[i, :a], tokens[i, :a]) and 0 <= out[i, a] < 640
    say("sampled: %d of 72 drafts accepted" % taken)
