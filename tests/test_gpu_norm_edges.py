"""pn_residual_norm where a gate is far below zero."""
import numpy as np
import pytest

import step_ref as R
from test_gpu_norm import EPS, call, host, make

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
