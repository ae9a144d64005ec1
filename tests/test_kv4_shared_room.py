"""pn_kv4_attn_shared_workspace on the CPU: what a caller keeps for its largest
call serves every smaller one."""
import itertools

import pytest

from bit_quantized_decode_pn3t_amd import _binding as B

FAKE = 0x10000  # never dereferenced


def cache(page, heads, dim):
    return B.KV4Cache(FAKE, 4, page, heads, dim)


def size(c, q_heads, **kw):
    return B.pn_kv4_attn_shared_workspace(c, q_heads, *[kw[k] for k in ("B", "G", "total_q", "max_q", "max_kv", "max_shared")])


AXES = dict(B=(1, 10, 11, 40, 64, 128, 300), G=(1, 2, 64, 65, 200), total_q=(1, 8, 40, 64, 297, 2048, 20000),
            max_q=(1, 2, 5, 9, 33, 64, 300, 2000), max_kv=(64, 1024, 1025, 20480), max_shared=(1, 4, 256, 400))


@pytest.mark.parametrize("page,heads,q_heads,dim", [(64, 8, 48, 128), (16, 16, 96, 64), (32, 4, 24, 256), (64, 1, 1, 64),
                                                    (16, 2, 32, 64)])
def test_room_for_smaller_calls(page, heads, q_heads, dim):
    """Along every size, with the others fixed: so of any two calls, the one that is larger in none needs no more."""
    c, names = cache(page, heads, dim), list(AXES)
    need = {at: size(c, q_heads, **{k: AXES[k][i] for k, i in zip(names, at)})
            for at in itertools.product(*(range(len(AXES[k])) for k in names))}
    assert all(need.values())
    for at, n in need.items():
        for k in range(len(names)):
            if at[k]:
                less = at[:k] + (at[k] - 1,) + at[k + 1:]
                assert need[less] <= n, (names, less, at, need[less], n)


def test_a_batch_that_shrinks():
    c = cache(64, 8, 128)
    most = size(c, 48, B=64, G=1, total_q=64, max_q=1, max_kv=20480, max_shared=256)
    for n in range(1, 64):
        assert size(c, 48, B=n, G=1, total_q=n, max_q=1, max_kv=20480, max_shared=256) <= most
    assert most <= 32 << 20
