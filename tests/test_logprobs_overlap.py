"""pn_logprobs on the CPU: outputs and workspace over inputs or each other are
refused, before any launch."""
import itertools

import pytest

from bit_quantized_decode_pn3t_amd import _binding as B

EINVAL = -1
MIB = 1 << 20
# never dereferenced: every call below fails its host checks
ARGS = dict(logits=MIB, row_type="f32", ld=1000, rows=40, V=990, scale=1.0, tokens=2 * MIB, ld_tok=3, n_tok=2, logp=3 * MIB,
            ld_lp=2, entropy=4 * MIB, K=5, top_ids=5 * MIB, top_logp=6 * MIB, ld_top=5, ws=7 * MIB, ws_bytes=8 * MIB)
OUT = ("logp", "entropy", "top_ids", "top_logp", "ws")


@pytest.mark.parametrize("out,other", [(a, b) for a, b in itertools.product(OUT, OUT + ("logits", "tokens")) if a != b])
def test_one_over_another(out, other):
    assert B.pn_logprobs(**dict(ARGS, **{out: ARGS[other]}), stream=0, check=False) == EINVAL


@pytest.mark.parametrize("kw", [
    dict(entropy=MIB + 39 * 4000 + 4 * 989), dict(entropy=MIB - 39 * 4),                  # the logits' last entry, and the first
    dict(logp=MIB + 4 * 989, ld_lp=1000), dict(top_ids=MIB + 4 * 996, ld_top=1000),       # columns that run into the row's
    dict(tokens=3 * MIB + 4, ld_tok=2), dict(top_logp=5 * MIB + 4, ld_top=5),
    dict(entropy=2 * MIB + 4 * 2 + 4 * 3 * 39 - 39 * 4 - 4),                                # ends in the last given token
])
def test_by_a_byte(kw):
    assert B.pn_logprobs(**dict(ARGS, **kw), stream=0, check=False) == EINVAL
