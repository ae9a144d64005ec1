"""pn_kv4_attn_shared on the CPU: refusals (status before any launch) and
workspace sizes."""
import pytest

from bit_quantized_decode_pn3t_amd import _binding as B

EINVAL, ESHAPE, EALIGN, EUNSUPPORTED = -1, -2, -3, -4
FAKE = 0x10000  # never dereferenced: every call below fails its host checks


def cache(pages=FAKE, num=4, page=16, heads=2, dim=64):
    return B.KV4Cache(pages, num, page, heads, dim)


ARGS = dict(q=FAKE, ldq=256, q_heads=4, q_start=FAKE, kv_len=FAKE, table=FAKE, ld_table=8, B=3, g_start=FAKE, prefix=FAKE,
            ld_prefix=4, shared=FAKE, G=1, total_q=3, max_q=1, max_kv=128, max_shared=4, scale=0.125, out=FAKE, ldo=256,
            ws=FAKE, ws_bytes=1 << 28)


@pytest.mark.parametrize("kw,status", [
    *[({k: None}, EINVAL) for k in ("q", "q_start", "kv_len", "table", "g_start", "prefix", "shared", "out", "ws")],
    *[({k: FAKE + 2}, EALIGN) for k in ("q_start", "kv_len", "table", "g_start", "prefix", "shared")],
    *[({k: FAKE + 8}, EALIGN) for k in ("q", "out", "ws")],
    (dict(ldq=260), EALIGN), (dict(ldo=260), EALIGN), (dict(ldq=248), ESHAPE), (dict(ldo=248), ESHAPE),
    (dict(q_heads=3), ESHAPE), (dict(q_heads=1), ESHAPE), (dict(B=0), ESHAPE), (dict(G=0), ESHAPE),
    (dict(total_q=-1), ESHAPE), (dict(max_q=0), ESHAPE), (dict(max_kv=0), ESHAPE), (dict(max_shared=0), ESHAPE),
    (dict(ld_table=7), ESHAPE), (dict(ld_prefix=3), ESHAPE), (dict(ws_bytes=3 * 4 * (4 * 64 + 8)), ESHAPE), (dict(ws_bytes=0), ESHAPE),
    (dict(scale=float("nan")), ESHAPE), (dict(scale=float("inf")), ESHAPE), (dict(scale=-float("inf")), ESHAPE),
    (dict(B=65536), EUNSUPPORTED), (dict(G=65536), EUNSUPPORTED), (dict(total_q=1 << 30), EUNSUPPORTED),
    (dict(total_q=1 << 28), EUNSUPPORTED), (dict(max_kv=1 << 30, ld_table=1 << 26), EUNSUPPORTED),
])
def test_checks(kw, status):
    assert B.pn_kv4_attn_shared(cache(), **dict(ARGS, **kw), stream=0, check=False) == status


@pytest.mark.parametrize("kw,status", [(dict(pages=None), EINVAL), (dict(page=20), ESHAPE), (dict(dim=80), ESHAPE),
                                       (dict(pages=FAKE + 8), EALIGN)])
def test_cache_checks(kw, status):
    assert B.pn_kv4_attn_shared(cache(**kw), **ARGS, stream=0, check=False) == status


def test_nothing_to_do_and_sizes():
    c = cache()
    assert B.pn_kv4_attn_shared(c, **dict(ARGS, total_q=0), stream=0, check=False) == 0
    size = B.pn_kv4_attn_shared_workspace
    assert size(c, 4, 3, 1, 3, 1, 128, 4) >= 3 * 4 * (4 * 64 + 8) + 12
    assert size(c, 4, 3, 1, 3, 1, 100000, 6000) > size(c, 4, 3, 1, 3, 1, 128, 4)  # room for splits
    for bad in ((3, 3, 1, 3, 1, 128, 4), (4, 0, 1, 3, 1, 128, 4), (4, 3, 0, 3, 1, 128, 4), (4, 3, 1, 3, 1, 128, 0),
                (4, 3, 1, 0, 1, 128, 4), (4, 3, 1, 1 << 30, 1, 128, 4)):
        assert size(c, *bad) == 0
    assert B.lib().pn_kv4_attn_shared_workspace(None, 4, 3, 1, 3, 1, 128, 4) == 0


@pytest.mark.parametrize("requests,groups,status", [(32767, 1, ESHAPE), (32768, 1, EUNSUPPORTED), (65535, 1, EUNSUPPORTED),
                                                    (4, 65535, EUNSUPPORTED)])
def test_more_items_than_a_launch_holds(requests, groups, status):
    """A workgroup of 512 threads to an item: 2^32 threads from 2^23 items on."""
    c = cache(heads=256)
    kw = dict(ARGS, ldq=16384, ldo=16384, q_heads=256, B=requests, G=groups, total_q=requests, ws_bytes=16)
    assert B.pn_kv4_attn_shared(c, **kw, stream=0, check=False) == status
    size = B.pn_kv4_attn_shared_workspace(c, 256, requests, groups, requests, 1, 128, 4)
    assert (size == 0) == (status == EUNSUPPORTED)
