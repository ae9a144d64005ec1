"""pn_logprobs against a plain 64-bit implementation: alternatives equal,
logarithms within bounds that count the fp32 roundings (tests/step_ref.py)."""
import numpy as np
import pytest

import step_ref as R
from gpu_util import say

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_quantized_decode_pn3t_amd import _binding as B  # noqa: E402

BIG = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield


def run(x, scale, tokens, K, pad=0, off=0, entropy=True):
    """x: numpy fp32 or fp16 [rows, V]; pad: elements behind a row; off: elements in front of the first."""
    rows, V = x.shape
    ld = V + pad
    flat = torch.full((off + rows * ld,), 1e4, dtype=torch.float16 if x.dtype == np.float16 else torch.float32, device="cuda")
    view = flat[off:].view(rows, ld)
    view[:, :V] = torch.from_numpy(x).cuda()
    tok = torch.from_numpy(np.ascontiguousarray(tokens, np.int32)).cuda()
    n = tok.shape[1]
    out = dict(logp=torch.full((rows, n + 1), 7.0, device="cuda"), entropy=torch.full((rows,), 7.0, device="cuda"),
               ids=torch.full((rows, K + 1), 7, dtype=torch.int32, device="cuda"),
               best=torch.full((rows, K + 1), 7.0, device="cuda"))
    need = B.pn_logprobs_workspace(rows, V, K)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")

    def go():
        B.pn_logprobs(view, "f16" if x.dtype == np.float16 else "f32", ld, rows, V, scale, tok, n, n, out["logp"], n + 1,
                      out["entropy"] if entropy else None, K, out["ids"], out["best"], K + 1, ws, need)
    go()
    torch.cuda.synchronize()
    assert (ws[need:] == 0xA5).all()
    got = {k: v.cpu().numpy() for k, v in out.items()}
    assert (got["logp"][:, n] == 7).all() and (got["ids"][:, K] == 7).all() and (got["best"][:, K] == 7).all()
    return got["logp"][:, :n], got["entropy"], got["ids"][:, :K], got["best"][:, :K], (go, out)


def near(got, want, bound):
    with np.errstate(invalid="ignore"):
        ok = (got == want) | (np.abs(got - want) <= bound)
    assert ok.all(), (got[~ok][:3], want[~ok][:3])


def check(got, x, scale, tokens, K, entropy=True):
    logp, H, ids, best, d, d_h = R.logprobs(x, scale, tokens, K)
    assert np.array_equal(got[2], ids)
    with np.errstate(invalid="ignore"):
        near(got[0], logp, d[:, None] + R.U * np.abs(logp))
        near(got[3], best, d[:, None] + R.U * np.abs(best))
    if entropy:
        near(got[1], H, d_h)


def case(rows, V, n, half=False, seed=0, spread=2.5, masked=0.0):
    g = np.random.default_rng([rows, V, seed])
    x = (spread * g.standard_normal((rows, V))).astype(np.float16 if half else np.float32)
    x[g.random((rows, V)) < masked] = -np.inf
    return x, g.integers(0, V, (rows, n))


@pytest.mark.parametrize("V", [1, 2, 5, 63, 64, 65, 1000, 1023, 1024, 1025, 4097, 32003, 62080])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("K", [0, 1, 20, 64])
def test_sizes(V, half, K):
    say("logprobs V=%d half=%d K=%d" % (V, half, K))
    x, tokens = case(5, V, 3, half)
    check(run(x, 1.25, tokens, K, pad=V % 3, off=V % 4), x, 1.25, tokens, K)


@pytest.mark.parametrize("rows,V,n,K", [(1, 248320, 1, 5), (70, 248320, 2, 20), (3000, 300, 0, 3), (517, 32003, 1, 64),
                                        (1, 1 << 20, 1, 8), (2, 3000, 700, 0)])
def test_shapes(rows, V, n, K):
    say("logprobs rows=%d V=%d n=%d K=%d" % (rows, V, n, K))
    x, tokens = case(rows, V, n)
    got = run(x, 0.7, tokens, K, pad=5)
    check(got, x, 0.7, tokens, K)
    assert B.pn_variant_name(B.pn_last_variant()) == "logprobs"


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("V", [700, 20011])
def test_masks(half, V):
    """Masked entries, rows with nothing, with one or two entries left, NaN, infinities, the type's lowest value."""
    x, tokens = case(10, V, 4, half, masked=0.9)
    low = np.finfo(x.dtype).min
    x[1] = -np.inf
    x[2] = -np.inf
    x[2, V // 2] = -3.0
    x[3] = np.nan
    x[4, ::3] = np.nan
    x[5, V // 3] = np.inf
    x[5, V // 3 + 5] = np.inf
    x[6] = low
    x[7] = low
    x[7, 5] = 2.0
    x[7, V - 1] = -np.inf
    x[8] = -np.inf
    x[8, V - 1] = 1.0
    x[8, 3] = 1.0
    tokens[:, 0] = -1
    tokens[:, 1] = V
    tokens[2, 2] = V // 2
    tokens[8, 2] = V - 1
    tokens[5, 2] = V // 3
    tokens[5, 3] = 2 ** 31 - 1
    check(run(x, 1.0, tokens, 20), x, 1.0, tokens, 20)


@pytest.mark.parametrize("V", [900, 30000])
def test_ties(V):
    """Equal entries go by the lower index: constant rows, few values, zeros of both signs."""
    g = np.random.default_rng(V)
    x = np.zeros((6, V), np.float32)
    x[1] = -4.5
    x[2] = g.integers(0, 3, V)
    x[3] = np.where(g.random(V) < 0.5, 0.0, -0.0)
    x[4] = np.sort(g.standard_normal(V))         # each better than all before
    x[5] = np.sort(g.standard_normal(V))[::-1]
    tokens = g.integers(0, V, (6, 2))
    for K in (1, 17, 64):
        check(run(x, 1.0, tokens, K), x, 1.0, tokens, K)


@pytest.mark.parametrize("spread,scale", [(40.0, 1.0), (1000.0, 2.0), (1e-3, 1.0), (1.0, 2.0 ** -64), (1e-6, 2.0 ** 64),
                                          (1e30, 1e-30)])
def test_far_values(spread, scale):
    """All but certain and all but even rows."""
    g = np.random.default_rng(3)
    x = (spread * g.standard_normal((7, 9000))).astype(np.float32)
    tokens = g.integers(0, 9000, (7, 2))
    tokens[:, 0] = x.argmax(1)
    check(run(x, scale, tokens, 5), x, scale, tokens, 5)


def test_certain_rows_keep_the_rest():
    """ln p of an entry at 1 - 1e-9 is -1e-9, not 0."""
    x = np.full((1, 5000), -40.0, np.float32)
    x[0, 77] = 0.0
    x[0, 78] = -20.0
    got = run(x, 1.0, np.array([[77, 78]]), 2)
    S1 = np.exp(-20.0) + 4998 * np.exp(-40.0)
    # the weight of one entry and its exponent: (20 * 3 + 44) half steps of S - 1
    assert abs(got[0][0, 0] + np.log1p(S1)) <= 110 * R.U * S1
    assert abs(got[1][0] - (np.log1p(S1) + (20 * np.exp(-20.0) + 40 * 4998 * np.exp(-40.0)) / (1 + S1))) <= 600 * R.U * 21 * S1


def test_without_parts_stream_and_graph():
    x, tokens = case(40, 33000, 2)
    check(run(x, 1.0, tokens, 3, entropy=False), x, 1.0, tokens, 3, entropy=False)
    *got, (go, out) = run(x, 1.0, tokens, 12)
    first = {k: v.clone() for k, v in out.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        go()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            go()
    for _ in range(3):
        for v in out.values():
            v.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for k, v in out.items():
            assert torch.equal(v, first[k]), k


def test_offsets_past_32_bits():
    """Rows of fp16 that lie 2^31 elements apart."""
    V, ld = 5000, (1 << 31) + 1
    buf = torch.empty(ld + V, dtype=torch.float16, device="cuda")
    x, tokens = case(2, V, 2, True)
    for r in range(2):
        buf[r * ld:r * ld + V] = torch.from_numpy(x[r]).cuda()
    tok = torch.from_numpy(tokens.astype(np.int32)).cuda()
    logp, H = torch.zeros(2, 2, device="cuda"), torch.zeros(2, device="cuda")
    ids, best = torch.zeros(2, 4, dtype=torch.int32, device="cuda"), torch.zeros(2, 4, device="cuda")
    ws = torch.empty(B.pn_logprobs_workspace(2, V, 4), dtype=torch.uint8, device="cuda")
    B.pn_logprobs(buf, "f16", ld, 2, V, 1.0, tok, 2, 2, logp, 2, H, 4, ids, best, 4, ws, ws.numel())
    check([t.cpu().numpy() for t in (logp, H, ids, best)], x, 1.0, tokens, 4)


def test_more_rows_than_a_launch_holds():
    """A row to 256 threads, less than 2^32 threads to a launch."""
    rows, V, K = (1 << 24) + 5, 3, 2
    x = torch.randn((rows, V), dtype=torch.float32, device="cuda")
    tok = torch.randint(0, V, (rows, 1), dtype=torch.int32, device="cuda")
    logp, H, best = (torch.full(s, 7.0, device="cuda") for s in ((rows, 1), (rows,), (rows, K)))
    ids = torch.full((rows, K), 7, dtype=torch.int32, device="cuda")
    need = B.pn_logprobs_workspace(rows, V, K)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    B.pn_logprobs(x, "f32", V, rows, V, 1.0, tok, 1, 1, logp, 1, H, K, ids, best, K, ws, need)
    torch.cuda.synchronize()
    for at in (0, (1 << 24) - 100, rows - 200):
        cut = slice(at, at + 200)
        check([t[cut].cpu().numpy() for t in (logp, H, ids, best)], x[cut].cpu().numpy(), 1.0, tok[cut].cpu().numpy(), K)
