"""pn_kv4_attn_shared with more than 64 groups, which a workgroup's waves search
together, and prefixes long enough for several parts an item."""
import numpy as np
import pytest

from gpu_util import say
from test_gpu_kv4_shared import run

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield


# A part has eight steps of 32 tokens at least: of few groups 300 tokens are 2 parts, 3000 are 12.
@pytest.mark.parametrize("dim,page,heads,group", [(64, 16, 1, 2), (64, 32, 2, 8), (128, 32, 1, 3), (256, 64, 1, 2)])
@pytest.mark.parametrize("groups", [65, 130, 600])
def test_prefixes_in_parts(dim, page, heads, group, groups):
    say("shared dim=%d page=%d heads=%d x %d groups=%d" % (dim, page, heads, group, groups))
    g = np.random.default_rng([dim, groups])
    sizes = [int(n) for n in g.integers(0, 3, groups)]
    tokens = np.exp(g.uniform(np.log(300), np.log(3000 if groups < 100 else 700), groups))
    pages = [int(t) // page if x else 0 for t, x in zip(tokens, g.random(groups) < 0.85)]
    n = sum(sizes) + 5
    run([30, dim, groups], [1] * n, [int(t) for t in g.integers(1, 40, n)], sizes, pages, dim, page, heads, group, g0=2,
        own_columns=False)


def test_few_long_among_many():
    """One group has all the keys: its items are cut into as many parts as a long step allows."""
    pages = [1] * 90
    pages[0], pages[44], pages[89] = 180, 400, 90
    run(31, [1] * 95, [3] * 95, [1] * 90, pages, 64, 16, 2, 4, g0=3, own_columns=False)


def test_drafts_of_many_groups():
    """Several row tiles a group."""
    g = np.random.default_rng(32)
    run(32, [5] * 80, [int(t) for t in g.integers(5, 30, 80)], [1] * 80, [int(p) for p in g.integers(20, 90, 80)], 64, 16, 1,
        16, own_columns=False)
