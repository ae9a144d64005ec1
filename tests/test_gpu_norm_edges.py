"""pn_residual_norm where a gate is far below zero, and with arrays that lie
between each other's rows."""
import numpy as np
import pytest

import step_ref as R
from gpu_util import say
from test_gpu_norm import EPS, FILL, call, check, host, make, want

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield


@pytest.mark.parametrize("gate", ["sigmoid", "silu"])
@pytest.mark.parametrize("half", [False, True])
def test_shut_gates(gate, half):
    """z from -80 to the type's lowest value, and -inf (by its limit, 0), over a stream of zeros and another.

    Below -88 a gate's values stay under 88 * 2^-126, so that a factor of the added term may be off by
    as much; both sides' are bounded."""
    n = 256
    s = make(4, n, half=half, post=False, gate=gate, seed=1)
    z = np.array([-80.0, -87.9, -88.1, -95.0, -103.0, -104.5, -110.0, -1e3, -6e4, float(torch.finfo(s["kind"]).min)] +
                 ([] if half else [-1e9, -1e20, -1e30]))
    z = np.resize(z, (4, n))
    s["z"][:, :n] = torch.from_numpy(z).to("cuda", s["kind"])
    s["h"][:2, :n] = 0
    s["z"][3, 5] = float("-inf")
    call(s)
    torch.cuda.synchronize()
    z = host(s["z"], n)
    z[3, 5] = -1e30
    h, y = host(s["h"], n), host(s["y"], n)
    out, dh, x, dx = R.residual_norm(h, y, False, None, gate, z, s["scale"], None, host(s["pre_gain"], n), EPS)
    more = 2 * np.abs(y) * 0.7 * 88 * 2.0 ** -126 + 2.0 ** -126  # and the smallest normal number's step
    got = host(s["h_out"], n)
    assert (np.abs(got - out) <= dh + more).all(), (gate, float(np.abs(got - out).max()))
    # of x: the added term by way of 1 / sqrt(eps) at most
    got = host(s["x"], n)
    assert (np.abs(got - x) <= dx + 2 * more / np.sqrt(EPS)).all()


@pytest.mark.parametrize("n", [200, 1500])
def test_between_rows(n):
    """Vectors and one gate row in the gaps of the stream's rows; rows of other pitches in a gap."""
    say("norm between rows n=%d" % n)
    T = 5
    s = make(T, n, gate="silu", chan=True, one_gate=True)
    ref = want(s)
    w = (n + 15) // 16 * 16
    wide = torch.full((T, 3 * w), FILL, dtype=torch.float32, device="cuda")
    wide[:, :n] = s["h"][:, :n]
    for t, name in enumerate(("post_gain", "pre_gain", "chan")):
        wide[t, w:w + n] = s[name]
    wide[3, w:w + n] = s["z"][0, :n]
    before = wide.clone()
    # in place, so that the vectors stand between rows that are written
    call(s, h=wide, ldh=3 * w, h_out=wide, ldho=3 * w, post_gain=wide[0, w:], pre_gain=wide[1, w:], chan_scale=wide[2, w:],
         z=wide[3, w:], ldz=0)
    s["h_out"] = wide[:, :n]
    check(s, ref)
    torch.cuda.synchronize()
    assert torch.equal(wide[:, w:], before[:, w:])


def test_rows_of_other_pitches_in_a_gap():
    """All of a short fp16 output behind the first row of the stream."""
    T, n = 3, 32
    s = make(T, n, post=False)
    ref = want(s)
    wide = torch.full((T, 256), FILL, dtype=torch.float32, device="cuda")
    wide[:, :n] = s["h"][:, :n]
    x = wide[0, 64:].view(torch.float16)[:T * 40].view(T, 40)  # rows of 80 bytes between bytes 256 and 496 of 1024
    x.fill_(FILL)
    call(s, h=wide, ldh=256, x=x, ldx=40)
    s["x"] = x
    check(s, ref)
