"""The attention-side entry points on the CPU: refusals (status before any
launch), size helpers, the plain 64-bit implementations against the C oracle,
and the assembly of the new kernels."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import kv4_ref as R
from bit_quantized_decode_pn3t_amd import _binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_quantized_decode_pn3t_amd", "csrc")
EINVAL, ESHAPE, EALIGN, EUNSUPPORTED = -1, -2, -3, -4
FAKE = 0x10000  # never dereferenced: every call below fails its host checks


def test_page_bytes():
    assert B.pn_kv4_page_bytes(16, 1, 64) == 16 * 68
    assert B.pn_kv4_page_bytes(64, 4, 256) == 64 * 4 * 272
    for bad in ((8, 1, 64), (24, 1, 64), (512, 1, 64), (16, 0, 64), (16, 1, 96), (16, -1, 64)):
        assert B.pn_kv4_page_bytes(*bad) == 0


def cache(pages=FAKE, num=4, page=16, heads=2, dim=64):
    return B.KV4Cache(pages, num, page, heads, dim)


@pytest.mark.parametrize("kw,status", [
    (dict(pages=None), EINVAL), (dict(num=0), ESHAPE), (dict(page=20), ESHAPE), (dict(heads=0), ESHAPE),
    (dict(dim=80), ESHAPE), (dict(pages=FAKE + 8), EALIGN), (dict(heads=65536), EUNSUPPORTED),
])
def test_cache_checks(kw, status):
    c = cache(**kw)
    assert B.pn_kv4_load(c, FAKE, 1, FAKE, FAKE, stream=0, check=False) == status
    assert store(c) == status
    assert attn(c=c) == status
    assert B.lib().pn_kv4_load(None, FAKE, 1, FAKE, FAKE, 0) == EINVAL


def test_load_checks():
    c = cache()
    assert B.pn_kv4_load(c, None, 1, FAKE, FAKE, stream=0, check=False) == EINVAL
    assert B.pn_kv4_load(c, FAKE, 1, None, None, stream=0, check=False) == EINVAL
    assert B.pn_kv4_load(c, FAKE, -1, FAKE, FAKE, stream=0, check=False) == ESHAPE
    assert B.pn_kv4_load(c, FAKE + 4, 1, FAKE, FAKE, stream=0, check=False) == EALIGN
    assert B.pn_kv4_load(c, FAKE, 1, FAKE + 4, FAKE, stream=0, check=False) == EALIGN
    assert B.pn_kv4_load(c, FAKE, 1 << 50, FAKE, FAKE, stream=0, check=False) == EUNSUPPORTED
    assert B.pn_kv4_load(c, FAKE, 0, FAKE, FAKE, stream=0, check=False) == 0
    with pytest.raises(B.PNError):
        B.pn_kv4_load(c, None, 1, FAKE, FAKE, stream=0)


PLAN = dict(ctx_len=FAKE, new_len=FAKE, held=FAKE, B=4, free_pages=FAKE, num_free=9, page_size=16, table=FAKE,
            ld_table=8, max_pages=8, held_out=FAKE + 0x100000, q_start=FAKE, kv_len=FAKE, positions=FAKE, slots=FAKE,
            max_tokens=64, info=FAKE)


@pytest.mark.parametrize("kw,status", [
    *[({k: None}, EINVAL) for k, v in PLAN.items() if isinstance(v, int) and v >= FAKE],
    *[({k: PLAN[k] + 2}, EALIGN) for k, v in PLAN.items() if isinstance(v, int) and v >= FAKE],
    (dict(slots=FAKE + 4), EALIGN), (dict(held_out=FAKE), EINVAL), (dict(held_out=FAKE + 8), EINVAL),
    (dict(B=0), ESHAPE), (dict(num_free=-1), ESHAPE), (dict(page_size=17), ESHAPE), (dict(max_pages=0), ESHAPE),
    (dict(ld_table=7), ESHAPE), (dict(max_tokens=0), ESHAPE), (dict(B=8193), EUNSUPPORTED),
    (dict(max_tokens=1 << 31), EUNSUPPORTED),
])
def test_plan_checks(kw, status):
    assert B.pn_kv4_plan(**dict(PLAN, **kw), stream=0, check=False) == status


STORE = dict(T=1, q=FAKE, k=FAKE, v=FAKE, row_type="f32", ldq=256, ldk=128, ldv=128, q_heads=4, q_gain=FAKE,
             k_gain=FAKE, eps=1e-6, inv_freq=FAKE, rot=64, pairs=False, positions=FAKE, slots=FAKE, q_out=FAKE, ldo=256)


def store(c, **kw):
    return B.pn_kv4_store(c, **dict(STORE, **kw), stream=0, check=False)


@pytest.mark.parametrize("kw,status", [
    (dict(positions=None), EINVAL), (dict(q=None, k=None, v=None), EINVAL), (dict(k=None), EINVAL),
    (dict(v=None), EINVAL), (dict(slots=None), EINVAL), (dict(q_out=None), EINVAL), (dict(inv_freq=None), EINVAL),
    (dict(row_type="bf16"), EINVAL), (dict(T=-1), ESHAPE), (dict(rot=-16), ESHAPE), (dict(rot=80), ESHAPE),
    (dict(eps=-1.0), ESHAPE), (dict(eps=float("nan")), ESHAPE), (dict(q_heads=0), ESHAPE), (dict(ldq=255), ESHAPE),
    (dict(ldo=255), ESHAPE), (dict(ldk=127), ESHAPE), (dict(ldv=127), ESHAPE), (dict(q=FAKE + 4), EALIGN),
    (dict(k=FAKE + 8), EALIGN), (dict(v=FAKE + 8), EALIGN), (dict(q_out=FAKE + 2), EALIGN),
    (dict(q_gain=FAKE + 4), EALIGN), (dict(k_gain=FAKE + 4), EALIGN), (dict(inv_freq=FAKE + 2), EALIGN),
    (dict(positions=FAKE + 2), EALIGN), (dict(slots=FAKE + 4), EALIGN), (dict(ldq=258), EALIGN),
    (dict(ldk=130), EALIGN), (dict(ldv=130), EALIGN), (dict(ldo=260), EALIGN), (dict(row_type="f16", ldk=132), EALIGN),
    (dict(rot=24), EUNSUPPORTED), (dict(T=0), 0),
])
def test_store_checks(kw, status):
    assert store(cache(), **kw) == status


ATTN = dict(q=FAKE, ldq=256, q_heads=4, q_start=FAKE, kv_len=FAKE, table=FAKE, ld_table=8, B=3, total_q=5, max_q=2,
            max_kv=100, scale=0.125, window=0, sinks=0, out=FAKE, ldo=256, ws=None, ws_bytes=0)


def attn(c=None, **kw):
    return B.pn_kv4_attn(c or cache(), **dict(ATTN, **kw), stream=0, check=False)


@pytest.mark.parametrize("kw,status", [
    *[({k: None}, EINVAL) for k in ("q", "q_start", "kv_len", "table", "out")], (dict(ws_bytes=16), EINVAL),
    (dict(q_heads=3), ESHAPE), (dict(q_heads=0), ESHAPE), (dict(q_heads=1), ESHAPE), (dict(B=0), ESHAPE),
    (dict(total_q=-1), ESHAPE), (dict(max_q=0), ESHAPE), (dict(max_kv=0), ESHAPE), (dict(sinks=-1), ESHAPE),
    (dict(ldq=255), ESHAPE), (dict(ldo=255), ESHAPE), (dict(ld_table=6), ESHAPE), (dict(q=FAKE + 8), EALIGN),
    (dict(out=FAKE + 8), EALIGN), (dict(ldq=260), EALIGN), (dict(ldo=260), EALIGN), (dict(q_start=FAKE + 2), EALIGN),
    (dict(kv_len=FAKE + 2), EALIGN), (dict(table=FAKE + 2), EALIGN), (dict(ws=FAKE + 8, ws_bytes=16), EALIGN),
    (dict(B=65536), EUNSUPPORTED), (dict(max_kv=1 << 31, ld_table=1 << 28), EUNSUPPORTED),
    (dict(total_q=1 << 31), EUNSUPPORTED), (dict(total_q=0), 0),
])
def test_attn_checks(kw, status):
    assert attn(**kw) == status


def test_attn_workspace_sizes():
    c = cache(heads=4, dim=128, num=1000)
    one = B.pn_kv4_attn_workspace(c, 24, 1, 1, 1, 16384)
    assert 0 < one < 64 << 20
    assert B.pn_kv4_attn_workspace(c, 24, 1, 1, 1, 16) == 0  # nothing to split
    assert B.pn_kv4_attn_workspace(c, 25, 1, 1, 1, 16384) == 0  # refused sizes
    assert B.pn_kv4_attn_workspace(c, 24, 1, 0, 1, 16384) == 0


SPEC = dict(target=FAKE, ldt=100, draft=FAKE, ldd=100, tokens=FAKE, ld_tok=3, n_draft=FAKE, u=FAKE, ldu=4, B=2, k=3,
            V=100, out=FAKE, ld_out=4, accepted=FAKE, ws=FAKE, ws_bytes=1 << 20)


@pytest.mark.parametrize("kw,status", [
    *[({k: None}, EINVAL) for k in ("target", "tokens", "u", "out", "accepted", "ws")],
    *[({k: FAKE + 2}, EALIGN) for k in ("target", "draft", "tokens", "n_draft", "u", "out", "accepted")],
    (dict(ws=FAKE + 4), EALIGN), (dict(B=0), ESHAPE), (dict(k=-1), ESHAPE), (dict(V=0), ESHAPE),
    (dict(ldt=99), ESHAPE), (dict(ldd=99), ESHAPE), (dict(ld_tok=2), ESHAPE), (dict(ldu=3), ESHAPE),
    (dict(ld_out=3), ESHAPE), (dict(ws_bytes=8), ESHAPE), (dict(B=65536, ws_bytes=1 << 40), EUNSUPPORTED),
    (dict(k=1025, ld_tok=2000, ldu=2000, ld_out=2000), EUNSUPPORTED),
])
def test_spec_checks(kw, status):
    assert B.pn_spec_verify(**dict(SPEC, **kw), stream=0, check=False) == status


def test_spec_workspace_sizes():
    assert B.pn_spec_workspace(0, 100) == 0
    assert B.pn_spec_workspace(3, 0) == 0
    assert B.pn_spec_workspace(3, 100) >= 3 * 16
    assert B.pn_spec_workspace(1, 1 << 31) == 0


def test_struct_sizes():
    """The ctypes structures match the header's (natural alignment on x86-64)."""
    assert ctypes.sizeof(B.pn_kv4_cache) == 24
    assert ctypes.sizeof(B.pn_kv4_store_desc) == 136


# ---- the plain implementations -------------------------------------------
def test_ref_quantizer_is_the_oracles():
    g = np.random.default_rng(1)
    y = (g.standard_normal((64, 256)) * np.exp(2 * g.standard_normal((64, 1)))).astype(np.float32)
    y[3, :64] = 0
    y[4, 5], y[4, 9] = -7, 7  # equal magnitudes: the first gives the sign
    y[5, :64] = np.arange(-32, 32) / 4  # quotients on ties
    d0, n0 = R.quantize(y)
    d1, n1 = R.pnref_codes(y)
    assert np.array_equal(d0.view(np.uint16), d1.view(np.uint16))
    assert np.array_equal(n0, n1)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_ref_layout_round_trip(dim):
    """Every place of a page is written once, and reads back."""
    g = np.random.default_rng(dim)
    page, heads = 16, 2
    pages = np.zeros((2, R.page_bytes(page, heads, dim)), np.uint8)
    want = {}
    for slot in range(2 * page):
        for side in "kv":
            d = g.standard_normal((heads, dim // 64)).astype(np.float16)
            n = g.integers(0, 16, (heads, dim))
            R.put(pages, page, heads, dim, slot, side, d, n)
            want[slot, side] = R.value(d, n)
    k, v = R.get(pages, page, heads, dim, np.arange(2 * page))
    for slot in range(2 * page):
        assert np.array_equal(k[slot], want[slot, "k"]) and np.array_equal(v[slot], want[slot, "v"])


# ---- the kernels' assembly -----------------------------------------------
HIPCC = "/opt/rocm/bin/hipcc"


@pytest.mark.skipif(not os.path.exists(HIPCC) and shutil.which("hipcc") is None, reason="no hipcc")
@pytest.mark.parametrize("src", ["pn_kv4_plan.hip", "pn_kv4_store.hip", "pn_kv4_attn.hip", "pn_spec.hip"])
def test_assembly(tmp_path, src):
    """No packed fp32 arithmetic, no L2 write-back or invalidation."""
    out = tmp_path / (src + ".s")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "--cuda-device-only", "-S", "-Xclang",
                    "-target-feature", "-Xclang", "-packed-fp32-ops", "-I" + os.path.join(ROOT, "include"), "-o",
                    str(out), os.path.join(CSRC, src)], check=True, capture_output=True)
    asm = out.read_text()
    assert "s_endpgm" in asm
    bad = re.findall(r"^\s*(?:v_pk_(?:add|mul|fma)_f32|buffer_wbl2|buffer_inv)\b.*$", asm, re.M)
    assert bad == []
    if src == "pn_kv4_attn.hip":
        assert len(re.findall(r"^\s*v_mfma_f32_16x16x32_f16", asm, re.M)) > 100
