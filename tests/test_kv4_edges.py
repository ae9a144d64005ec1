"""Refusals of the attention-side entry points at their edges, on the CPU: every
call here fails its host checks before any launch."""
import pytest

from bit_quantized_decode_pn3t_amd import _binding as B

EINVAL, ESHAPE, EALIGN, EUNSUPPORTED = -1, -2, -3, -4
BASE = 0x100000  # never dereferenced

# what a plan reads and writes, and its bytes for 5 requests of 4 columns in rows of 7, 9 free pages and 33 tokens
READ = dict(ctx_len=20, new_len=20, held=20, free_pages=36)
WRITTEN = dict(table=4 * (4 * 7 + 4), held_out=20, q_start=24, kv_len=20, positions=132, slots=264, info=8)


def plan(**kw):
    place = {k: BASE + 0x1000 * i for i, k in enumerate([*READ, *WRITTEN])}
    place.update(kw)
    return B.pn_kv4_plan(B=5, num_free=9, page_size=16, ld_table=7, max_pages=4, max_tokens=33, stream=0, check=False,
                         **place)


@pytest.mark.parametrize("out", WRITTEN)
@pytest.mark.parametrize("other", [*READ, *WRITTEN])
def test_plan_refuses_outputs_over_other_arrays(out, other):
    if out == other:
        return
    at = BASE + 0x80000
    size = {**READ, **WRITTEN}
    last = 8 if "slots" in (out, other) else 4
    for shift in (0, size[other] - last, last - size[out]):  # the same place, its last word, up to its first
        shift = shift // last * last
        assert plan(**{other: at, out: at + shift}) == EINVAL, (out, other, shift)
