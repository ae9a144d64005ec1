"""pn_residual_norm and pn_logprobs on the CPU: refusals (status before any
launch), struct and workspace sizes."""
import ctypes

import pytest

from bit_quantized_decode_pn3t_amd import _binding as B

EINVAL, ESHAPE, EALIGN, EUNSUPPORTED = -1, -2, -3, -4
FAKE = 0x10000  # never dereferenced: every call below fails its host checks
NORM = dict(T=4, n=64, h=FAKE, ldh=64, y=2 * FAKE, ldy=64, row_type="f32", gate="silu", z=3 * FAKE, ldz=64, post=True,
            post_gain=4 * FAKE, scale=1.0, chan_scale=5 * FAKE, pre_gain=6 * FAKE, eps=1e-6, h_out=7 * FAKE, ldho=64,
            x=8 * FAKE, ldx=64)
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("kw,status", [
    (dict(h=None), EINVAL), (dict(h_out=None, x=None), EINVAL), (dict(row_type="bf16"), EINVAL),
    (dict(gate="tanh"), EINVAL), (dict(gate=4), EINVAL), (dict(z=None), EINVAL), (dict(gate="none"), EINVAL),
    (dict(post=False), EINVAL), (dict(y=None), EINVAL),
    (dict(y=None, gate="none", z=None, post=False, post_gain=None), EINVAL),  # chan_scale without y
    (dict(T=-1), ESHAPE), (dict(n=0), ESHAPE), (dict(scale=INF), ESHAPE), (dict(scale=NAN), ESHAPE),
    (dict(eps=-1e-6), ESHAPE), (dict(eps=NAN), ESHAPE), (dict(eps=INF), ESHAPE),
    *[({k: 60}, ESHAPE) for k in ("ldh", "ldy", "ldz", "ldho", "ldx")],
    *[({k: 66}, EALIGN) for k in ("ldh", "ldy", "ldz", "ldho")], (dict(ldx=68), EALIGN),
    (dict(row_type="f16", ldy=68), EALIGN), (dict(row_type="f16", ldz=68), EALIGN),
    *[({k: NORM[k] + 8}, EALIGN) for k in ("h", "y", "z", "post_gain", "chan_scale", "pre_gain", "h_out", "x")],
    (dict(n=32769, **{k: 32776 for k in ("ldh", "ldy", "ldz", "ldho", "ldx")}), EUNSUPPORTED),
    (dict(T=1 << 31), EUNSUPPORTED),
    # outputs over inputs or each other
    *[(dict(h_out=NORM[k]), EINVAL) for k in ("y", "z", "post_gain", "chan_scale", "pre_gain", "x")],
    *[(dict(x=NORM[k]), EINVAL) for k in ("h", "y", "z", "post_gain", "chan_scale", "pre_gain")],
    (dict(h_out=FAKE + 16), EINVAL), (dict(h_out=FAKE, ldho=68), EINVAL),
    (dict(h=FAKE, h_out=FAKE + 128, ldh=64, ldho=64), EINVAL),  # columns that overlap a row's end
])
def test_norm_checks(kw, status):
    assert B.pn_residual_norm(**dict(NORM, **kw), stream=0, check=False) == status


def test_norm_accepts_nothing_to_do():
    assert B.pn_residual_norm(**dict(NORM, T=0), stream=0, check=False) == 0
    assert B.pn_residual_norm(**dict(NORM, T=0, h_out=FAKE), stream=0, check=False) == 0  # in place
    assert B.lib().pn_residual_norm(None, None) == EINVAL
    with pytest.raises(B.PNError):
        B.pn_residual_norm(**dict(NORM, n=0), stream=0)


LOGP = dict(logits=FAKE, row_type="f32", ld=1000, rows=4, V=1000, scale=1.0, tokens=FAKE, ld_tok=2, n_tok=2, logp=FAKE,
            ld_lp=2, entropy=FAKE, K=5, top_ids=FAKE, top_logp=FAKE, ld_top=5, ws=FAKE, ws_bytes=1 << 20)


@pytest.mark.parametrize("kw,status", [
    *[({k: None}, EINVAL) for k in ("logits", "tokens", "logp", "top_ids", "top_logp", "ws")],
    (dict(row_type="bf16"), EINVAL), (dict(rows=-1), ESHAPE), (dict(V=0), ESHAPE), (dict(n_tok=-1), ESHAPE),
    (dict(K=-1), ESHAPE), (dict(ld=999), ESHAPE), (dict(ld_tok=1), ESHAPE), (dict(ld_lp=1), ESHAPE),
    (dict(ld_top=4), ESHAPE), (dict(scale=0.0), ESHAPE), (dict(scale=-1.0), ESHAPE), (dict(scale=NAN), ESHAPE),
    (dict(scale=INF), ESHAPE), (dict(scale=1e30), ESHAPE), (dict(ws_bytes=64), ESHAPE),
    *[({k: FAKE + 2}, EALIGN) for k in ("logits", "tokens", "logp", "entropy", "top_ids", "top_logp", "ws")],
    (dict(logits=FAKE + 1, row_type="f16"), EALIGN), (dict(ws=FAKE + 4), EALIGN),
    (dict(K=65, ld_top=65), EUNSUPPORTED), (dict(V=1 << 31, ld=1 << 31), EUNSUPPORTED),
    (dict(rows=1 << 31), EUNSUPPORTED), (dict(rows=1 << 30, V=4096, ld=4096), EUNSUPPORTED),
])
def test_logprobs_checks(kw, status):
    assert B.pn_logprobs(**dict(LOGP, **kw), stream=0, check=False) == status


def test_logprobs_sizes():
    assert B.pn_logprobs(**dict(LOGP, rows=0), stream=0, check=False) == 0
    assert B.pn_logprobs_workspace(0, 10, 5) == 0 and B.pn_logprobs_workspace(1, 0, 5) == 0
    assert B.pn_logprobs_workspace(1, 10, 65) == 0 and B.pn_logprobs_workspace(1, 10, -1) == 0
    assert 0 < B.pn_logprobs_workspace(1, 10, 0) < B.pn_logprobs_workspace(1, 10, 64)
    # what a caller keeps for the largest call serves smaller ones
    most = B.pn_logprobs_workspace(512, 248320, 20)
    assert most <= 64 << 20
    for rows in (1, 7, 100, 511):
        assert B.pn_logprobs_workspace(rows, 248320, 20) <= most


def test_struct_size():
    assert ctypes.sizeof(B.pn_residual_norm_desc) == 8 * 8 + 7 * 8 + 5 * 4 + 4
