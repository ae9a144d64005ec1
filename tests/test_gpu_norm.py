"""pn_residual_norm against a plain 64-bit implementation, within bounds that
count its fp32 roundings and the one fp16 rounding (tests/step_ref.py)."""
import numpy as np
import pytest

import step_ref as R
from gpu_util import say

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_quantized_decode_pn3t_amd import _binding as B  # noqa: E402

EPS = 1e-6
FILL = -77.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield


def rows(a, kind, pad=8):
    """Device rows [T, ld], ld past n by `pad` to twice that, the gap filled."""
    T, n = a.shape
    t = torch.full((T, (n + 7) // 8 * 8 + pad), FILL, dtype=kind, device="cuda")
    t[:, :n] = torch.from_numpy(a).to("cuda", kind)
    return t


def make(T, n, half=False, post=True, gate="none", chan=False, gains=True, one_gate=False, seed=0):
    g = np.random.default_rng([T, n, seed])
    kind = torch.float16 if half else torch.float32
    s = dict(T=T, n=n, post=post, gate=gate, kind=kind, scale=0.7)
    s["h"] = rows((3 * np.exp(0.7 * g.standard_normal(n)) * g.standard_normal((T, n))).astype(np.float32), torch.float32)
    s["y"] = rows(1.7 * g.standard_normal((T, n)), kind)
    s["z"] = rows(2 * g.standard_normal((1 if one_gate else T, n)), kind) if gate != "none" else None
    s["ldz"] = 0 if one_gate or gate == "none" else s["z"].shape[1]

    def vec(a):
        return torch.from_numpy(a.astype(np.float32)).cuda()
    s["post_gain"] = vec(1 + 0.2 * g.standard_normal(n)) if post and gains else None
    s["pre_gain"] = vec(1 + 0.2 * g.standard_normal(n)) if gains else None
    s["chan"] = vec(0.1 + g.random(n)) if chan else None
    s["h_out"] = rows(np.zeros((T, n)), torch.float32, 16)
    s["x"] = rows(np.zeros((T, n)), torch.float16, 24)
    return s


def call(s, **kw):
    a = dict(T=s["T"], n=s["n"], h=s["h"], ldh=s["h"].shape[1], y=s["y"], ldy=s["y"].shape[1],
             row_type="f16" if s["kind"] == torch.float16 else "f32", gate=s["gate"], z=s["z"], ldz=s["ldz"],
             post=s["post"], post_gain=s["post_gain"], scale=s["scale"], chan_scale=s["chan"], pre_gain=s["pre_gain"],
             eps=EPS, h_out=s["h_out"], ldho=s["h_out"].shape[1], x=s["x"], ldx=s["x"].shape[1])
    a.update(kw)
    B.pn_residual_norm(**a)


def host(t, n):
    return None if t is None else t[:, :n].double().cpu().numpy() if t.dim() == 2 else t.double().cpu().numpy()


def want(s, h=None):
    n = s["n"]
    return R.residual_norm(host(s["h"], n) if h is None else h, host(s["y"], n) if s["y"] is not None else None, s["post"],
                           host(s["post_gain"], n), s["gate"], host(s["z"], n), s["scale"], host(s["chan"], n),
                           host(s["pre_gain"], n), EPS)


def check(s, ref, h=True, x=True):
    n = s["n"]
    torch.cuda.synchronize()
    for name, on, at in (("h_out", h, 0), ("x", x, 2)):
        got = s[name].double().cpu().numpy()
        if not on:
            assert (got[:, :n] == 0).all()
            continue
        err = np.abs(got[:, :n] - ref[at])
        assert (err <= ref[at + 1]).all(), (name, float((err / ref[at + 1]).max()))
        assert (got[:, n:] == FILL).all(), name


@pytest.mark.parametrize("n", [1, 3, 4, 63, 64, 255, 256, 257, 768, 1024, 1027, 2048, 2050, 5120, 6144, 8192, 8195,
                               12288, 17408, 32765, 32768])
@pytest.mark.parametrize("T", [1, 5])
def test_widths(n, T):
    say("norm T=%d n=%d" % (T, n))
    s = make(T, n, half=n % 2 == 1, chan=n % 3 == 0, gate=("none", "silu")[T == 5])
    call(s)
    check(s, want(s))
    assert B.pn_variant_name(B.pn_last_variant()) == "residual_norm"


@pytest.mark.parametrize("n", [130, 1500, 9000])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("post,gate,chan,gains,one_gate", [
    (False, "none", False, True, False), (True, "none", True, False, False), (False, "plain", False, True, True),
    (True, "plain", True, True, False), (False, "sigmoid", True, False, False), (True, "sigmoid", False, True, True),
    (True, "silu", False, False, False),
])
def test_forms(n, half, post, gate, chan, gains, one_gate):
    say("norm n=%d half=%d post=%d gate=%s" % (n, half, post, gate))
    s = make(67, n, half, post, gate, chan, gains, one_gate)
    call(s)
    check(s, want(s))


def test_many_rows():
    s = make(3001, 200, gate="sigmoid")
    call(s)
    check(s, want(s))


@pytest.mark.parametrize("n", [200, 5120])
def test_parts_and_places(n):
    """No block's output; only one output; in place; columns of one buffer."""
    say("norm parts n=%d" % n)
    s = make(9, n, post=False)
    s["y"], y = None, s["y"]
    none = dict(y=None, ldy=0)
    s0 = dict(s, y=y)
    call(s0, **none)
    check(s, want(s))
    s["h_out"][:, :n] = 0
    call(s0, h_out=None, ldho=0, **none)
    check(s, want(s), h=False)
    s = make(9, n)
    ref = want(s)
    call(s, x=None, ldx=0)
    check(s, ref, x=False)
    call(s, h_out=s["h"], ldho=s["h"].shape[1])
    s["h_out"] = s["h"][:, :n]
    check(s, ref)
    # stream and block output side by side, written next to each other
    s = make(9, n)
    ref = want(s)
    w = s["h"].shape[1]
    wide = torch.cat((s["h"], s["y"], torch.full_like(s["h"], FILL)), 1)
    call(s, h=wide, ldh=3 * w, y=wide[:, w:], ldy=3 * w, h_out=wide[:, 2 * w:], ldho=3 * w)
    s["h_out"] = wide[:, 2 * w:]
    check(s, ref)


def test_values_at_the_edges():
    """A stream of zeros, far values, entries without a number: by the formula, row by row."""
    n = 640
    s = make(6, n, gate="sigmoid")
    s["h"][0, :n] = 0
    s["y"][0, :n] = 0                     # 0 * 1/sqrt(eps)
    s["z"][1, :n] = -200                  # a closed gate
    s["z"][2, :n] = 200
    s["h"][3, :n] *= 1e15                 # squares near the end of fp32
    s["h"][4, :n] *= 1e-30
    s["y"][4, :n] *= 1e-30                # squares below it: eps alone
    s["h"][5, 7] = float("nan")
    call(s)
    h = host(s["h"], n)
    ref = R.residual_norm(*[a[:5] if a is not None and a.ndim == 2 else a for a in (h, host(s["y"], n))], True,
                          host(s["post_gain"], n), "sigmoid", host(s["z"], n)[:5], s["scale"], None,
                          host(s["pre_gain"], n), EPS)
    torch.cuda.synchronize()
    for got, at in ((s["h_out"], 0), (s["x"], 2)):
        got = got[:, :n].double().cpu().numpy()
        # an underflow costs the smallest normal number's step
        assert (np.abs(got[:5] - ref[at]) <= ref[at + 1] + 2.0 ** -126).all()
        assert np.isnan(got[5]).any()
    assert s["x"][5, :n].isnan().all()


def test_row_is_the_same_whatever_the_batch():
    s = make(64, 5120, gate="silu")
    call(s)
    torch.cuda.synchronize()
    h, x = s["h_out"].clone(), s["x"].clone()
    for t in (0, 13, 63):
        one = dict(s, T=1, h=s["h"][t:t + 1], y=s["y"][t:t + 1], z=s["z"][t:t + 1])
        s["h_out"][:1] = 0
        call(one)
        torch.cuda.synchronize()
        assert torch.equal(s["h_out"][0, :5120], h[t, :5120]) and torch.equal(s["x"][0, :5120], x[t, :5120])


def test_stream_and_graph():
    s = make(33, 5120, gate="silu")
    call(s)
    torch.cuda.synchronize()
    h, x = s["h_out"].clone(), s["x"].clone()
    side = torch.cuda.Stream()
    s["h_out"].zero_(), s["x"].zero_()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call(s)
        side.synchronize()
        assert torch.equal(s["x"][:, :5120], x[:, :5120])
        with torch.cuda.graph(graph, stream=side):
            call(s)
    for _ in range(3):
        s["h_out"].zero_(), s["x"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s["h_out"][:, :5120], h[:, :5120]) and torch.equal(s["x"][:, :5120], x[:, :5120])


def test_offsets_past_32_bits():
    """The last of rows that lie 2^30 elements apart and more."""
    n, ld = 1024, (1 << 30) + 8
    buf = torch.empty(2 * ld + n, dtype=torch.float32, device="cuda")
    s = make(3, n, post=False)
    for t in range(3):
        buf[t * ld:t * ld + n] = s["h"][t, :n]
    call(s, h=buf, ldh=ld, h_out=buf, ldho=ld)
    ref = want(s)
    for t in range(3):
        s["h_out"][t, :n] = buf[t * ld:t * ld + n]
    check(s, ref)


def test_more_rows_than_a_launch_holds():
    """Four rows to 256 threads, less than 2^32 threads to a launch."""
    T, n = (1 << 26) + 7, 3
    h = torch.randn((T, 4), dtype=torch.float32, device="cuda")
    x = torch.full((T, 8), FILL, dtype=torch.float16, device="cuda")
    B.pn_residual_norm(T=T, n=n, h=h, ldh=4, y=None, ldy=0, row_type="f32", gate="none", z=None, ldz=0, post=False,
                       post_gain=None, scale=1.0, chan_scale=None, pre_gain=None, eps=EPS, h_out=None, ldho=0, x=x, ldx=8)
    torch.cuda.synchronize()
    for at in (0, (1 << 26) - 12, T - 300):
        part = host(h[at:at + 300], n)
        _, _, ref, bound = R.residual_norm(part, None, False, None, "none", None, 1.0, None, None, EPS)
        got = x[at:at + 300].double().cpu().numpy()
        assert (np.abs(got[:, :n] - ref) <= bound).all() and (got[:, n:] == FILL).all()
