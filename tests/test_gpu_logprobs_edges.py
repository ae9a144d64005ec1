"""pn_logprobs where one workgroup takes a whole row in several steps, and with
outputs side by side in one buffer."""
import numpy as np
import pytest

import step_ref as R
from gpu_util import say
from test_gpu_logprobs import near

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_quantized_decode_pn3t_amd import _binding as B  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield


def compare(got, x, scale, tokens, K, lane):
    """lane: entries of a lane's sum (step_ref counts 256; each further one is a rounding of the entropy's
    sum, whose terms add up to the entropy at most)."""
    logp, H, ids, best, d, d_h = R.logprobs(x, scale, tokens, K)
    d_h = d_h + max(0, lane - 256) * R.U * H
    assert np.array_equal(got[2], ids)
    with np.errstate(invalid="ignore"):
        near(got[0], logp, d[:, None] + R.U * np.abs(logp))
        near(got[3], best, d[:, None] + R.U * np.abs(best))
    near(got[1], H, d_h)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rows,V,K,masked", [(1500, 4097, 20, 0.0), (1100, 9001, 1, 0.5), (1030, 32003, 64, 0.9),
                                             (1100, 8192, 0, 0.0), (1024, 131072, 20, 0.0), (2000, 20011, 64, 0.0)])
def test_whole_rows(half, rows, V, K, masked):
    """More rows than workgroups that share rows: 4 a compute unit, of 256 at most."""
    say("logprobs whole rows=%d V=%d half=%d K=%d" % (rows, V, half, K))
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + V)
    x = torch.empty((rows, V), dtype=torch.float16 if half else torch.float32, device="cuda")
    for i in range(0, rows, 128):
        part = 2.5 * torch.randn((min(128, rows - i), V), generator=g, device="cuda")
        part[torch.rand(part.shape, generator=g, device="cuda") < masked] = float("-inf")
        x[i:i + 128] = part.to(x.dtype)
    # rows of nothing, sorted up and down, of one value, with what counts at the end
    x[3] = float("-inf")
    x[4] = float("nan")
    x[5] = x[5].sort().values
    x[6] = x[6].sort(descending=True).values
    x[7] = 1.5
    x[8, :V - 3] = float("-inf")
    x[9, ::2] = float("nan")
    x[10, V - 1] = float("inf")
    x[11, :V - 100] = -60.0
    tokens = torch.randint(0, V, (rows, 2), generator=g, dtype=torch.int32, device="cuda")
    tokens[:, 1] = V - 1
    out = [torch.full((rows, 2), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda"),
           torch.full((rows, K), 7, dtype=torch.int32, device="cuda"), torch.full((rows, K), 7.0, device="cuda")]
    need = B.pn_logprobs_workspace(rows, V, K)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    B.pn_logprobs(x, "f16" if half else "f32", V, rows, V, 0.8, tokens, 2, 2, out[0], 2, out[1], K, out[2] if K else None,
                  out[3] if K else None, K, ws, need)
    torch.cuda.synchronize()
    at = list(range(14)) + [rows // 2, rows - 2, rows - 1]
    compare([t[at].cpu().numpy() for t in out], x[at].cpu().numpy(), 0.8, tokens[at].cpu().numpy(), K, -(-V // 256))


def test_outputs_side_by_side():
    """All outputs in columns of one buffer, behind the row that they are of."""
    rows, V, K = 9, 700, 5
    g = np.random.default_rng(4)
    x = (2.5 * g.standard_normal((rows, V))).astype(np.float32)
    tokens = g.integers(0, V, (rows, 3))
    buf = torch.full((rows, 720), 1e4, device="cuda")
    buf[:, :V] = torch.from_numpy(x).cuda()
    ints = buf.view(torch.int32)
    ints[:, 700:703] = torch.from_numpy(tokens.astype(np.int32)).cuda()
    before = buf[:, :703].clone()
    H = torch.zeros(rows, device="cuda")
    need = B.pn_logprobs_workspace(rows, V, K)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    B.pn_logprobs(buf, "f32", 720, rows, V, 1.0, ints[:, 700:], 720, 3, buf[:, 703:], 720, H, K, ints[:, 706:], buf[:, 711:],
                  720, ws, need)
    torch.cuda.synchronize()
    assert torch.equal(buf[:, :703].view(torch.int32), before.view(torch.int32)) and (buf[:, 716:] == 1e4).all()
    compare([t.cpu().numpy() for t in (buf[:, 703:706], H, ints[:, 706:711], buf[:, 711:716])], x, 1.0, tokens, K, 3)
