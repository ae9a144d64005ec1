"""pn_kv4_attn_shared against a plain 64-bit implementation, which attends each
request over its prefix and its own keys at once, within kv4_ref's bound: the
two fp16 roundings, and fp32 sums (joining two of them adds six roundings to
the 64 that the bound counts beside the keys)."""
import numpy as np
import pytest

import kv4_ref as R
from gpu_util import dev, say, sync
from test_gpu_kv4 import i32, make_cache

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_quantized_decode_pn3t_amd import _binding as B  # noqa: E402

SHAPES = [(64, 16, 2, 1), (64, 64, 1, 16), (128, 16, 2, 6), (128, 256, 1, 3), (256, 32, 1, 6), (256, 16, 3, 2)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield


def run(seed, q_lens, tails, sizes, prefix_pages, dim, page, heads, group, scale=None, sharp=1.0,
        wild=False, holes=(), own_columns=True, g0=0, inside=(), max_shared=None, max_kv=None, spoil=True, gap=0):
    """Requests in groups of `sizes` (from request g0 on), the rest alone; tails: each one's own keys.
    inside: requests whose length is less than their prefix.  own_columns: table rows hold the prefix's pages too."""
    g = np.random.default_rng(seed)
    n, q_heads = len(q_lens), heads * group
    of = np.full(n, -1)
    start = [g0]
    for i, m in enumerate(sizes):
        of[start[-1]:start[-1] + m] = i
        start.append(start[-1] + m)
    most = max(max(prefix_pages), 1) if max_shared is None else max_shared
    ahead = np.array([min(max(prefix_pages[i], 0), most) if i >= 0 else 0 for i in of])
    kv = np.array([a * page + t for a, t in zip(ahead, tails)])
    for b, length in inside:
        kv[b] = length
    top = max(kv.max(), 1) if max_kv is None else max_kv
    width = max(-(-int(kv.max()) // page), -(-top // page), 1)
    need = [-(-int(k) // page) for k in kv]
    num_pages = sum(max(p, 0) for p in prefix_pages) + sum(need) + 2
    pages = make_cache(g, num_pages, page, heads, dim, wild)
    ids = list(g.permutation(num_pages))
    prefix = np.full((len(sizes), max(most, max(prefix_pages))), -1)
    for i, p in enumerate(prefix_pages):
        for c in range(max(p, 0)):
            prefix[i, c] = ids.pop()
    table = np.full((n, width), -1)
    for b in range(n):
        for c in range(need[b]):
            table[b, c] = prefix[of[b], c] if c < ahead[b] else ids.pop()
    if spoil:  # what lies behind a request's last token holds NaN and infinite scales
        r = dim // 64
        for b in range(n):
            if any(x == b for x, _ in inside) or need[b] <= ahead[b]:
                continue
            for t in range(kv[b], need[b] * page):
                for h in range(heads):
                    base = h * page * (dim + dim // 16) + page * dim
                    for side in (0, 2 * page * r):
                        o = base + side + 2 * r * (t % page)
                        pages[table[b, t // page], o:o + 2 * r] = np.tile([0x00, 0x7e if t % 2 else 0xfc], r)
    for what, row, col, entry in holes:
        if what == "prefix":
            prefix[row, col] = entry
            for b in np.nonzero(of == row)[0]:
                table[b, col] = entry
        else:
            table[row, col] = entry
    whole = table.copy()
    if not own_columns:
        for b in range(n):
            if not any(x == b for x, _ in inside):
                table[b, :ahead[b]] = -1
    q_start = np.concatenate(([0], np.cumsum(q_lens)))
    T = int(q_start[-1])
    scale = dim ** -0.5 if scale is None else scale
    ld = q_heads * dim + 8
    q = (g.standard_normal((T + gap, ld)) * sharp).astype(np.float16)
    cache = B.KV4Cache(dev(pages), num_pages, page, heads, dim)
    max_q = max(max(q_lens), 1)
    size = B.pn_kv4_attn_shared_workspace(cache, q_heads, n, len(sizes), T, max_q, top, most)
    ws = torch.full(((size + 15) // 16 * 4 + 64,), float("nan"), device="cuda")
    out = torch.full((T + gap, ld), 9.0, dtype=torch.float16, device="cuda")
    args = [cache, dev(q), ld, q_heads, i32(q_start), i32(kv), i32(table), width, n, i32(start), i32(prefix),
            prefix.shape[1], i32(prefix_pages), len(sizes), T, max_q, top, most, scale, out, ld, ws, size]
    B.pn_kv4_attn_shared(*args)
    sync()
    assert B.pn_variant_name(B.pn_last_variant()) == "kv4_attn_shared"
    assert ws[(size + 15) // 16 * 4:].isnan().all()
    got = out.cpu().numpy()
    again = torch.full_like(out, 9.0)
    args[19] = again
    B.pn_kv4_attn_shared(*args)
    sync()
    assert np.array_equal(got.view(np.uint16), again.cpu().numpy().view(np.uint16)), "two runs differ"
    assert (got[T:] == 9).all() and (got[:, q_heads * dim:] == 9).all()
    want, bound = R.attend(q[:T, :q_heads * dim].reshape(T, q_heads, dim).astype(np.float64), pages, page, heads, dim, q_start,
                           np.minimum(kv, top), whole, np.float64(np.float32(scale)), 0, 0, num_pages)
    got = got[:T, :q_heads * dim].reshape(want.shape).astype(np.float64)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0].tolist(), got[bad][:4], want[bad][:4], bound[bad][:4])
    return args, got


@pytest.mark.parametrize("dim,page,heads,group", SHAPES)
@pytest.mark.parametrize("members,q,pages", [(1, 1, 1), (3, 1, 7), (9, 1, 3), (4, 5, 9)])
def test_one_group(dim, page, heads, group, members, q, pages):
    say("shared dim=%d page=%d heads=%d x %d members=%d q=%d pages=%d" % (dim, page, heads, group, members, q, pages))
    g = np.random.default_rng([dim, members, pages])
    tails = [int(t) for t in g.integers(q, q + 40, members)]
    tails[0] = q
    run([1, dim, members], [q] * members, tails, [members], [max(1, pages * 16 // page)], dim, page, heads, group)


@pytest.mark.parametrize("dim,page,heads,group", SHAPES)
def test_groups_and_others(dim, page, heads, group):
    """Groups of several lengths, one without a prefix, one empty, requests of their own in front and behind."""
    g = np.random.default_rng([dim, 5])
    q = [1, 3, 1, 2, 1, 1, 0, 4, 1, 1]
    tails = [int(x) for x in g.integers(4, 150, 10)]
    run([2, dim], q, tails, [3, 2, 0, 2], [5, 2, 1, 0], dim, page, heads, group, g0=1, own_columns=False, gap=3)


@pytest.mark.parametrize("dim,page,heads,group", SHAPES)
def test_long_prefix(dim, page, heads, group):
    """Keys split over workgroups."""
    say("shared long dim=%d page=%d" % (dim, page))
    run([3, dim], [1, 2, 1], [70, 3, 200], [3], [3000 // page], dim, page, heads, group)


@pytest.mark.parametrize("dim,heads,group,members,q", [(64, 1, 16, 40, 1), (64, 2, 4, 12, 13), (128, 2, 6, 60, 1),
                                                       (128, 1, 3, 10, 11), (256, 1, 6, 30, 1), (256, 1, 2, 9, 8)])
def test_many_rows(dim, heads, group, members, q):
    """Enough queries in a group for the kernels of many rows, and of one whose last tile is part empty."""
    say("shared rows dim=%d rows=%d" % (dim, members * q * group))
    g = np.random.default_rng([dim, members])
    run([4, dim], [q] * members, [int(t) for t in g.integers(q, q + 60, members)], [members], [1504 // 32], dim, 32, heads,
        group, own_columns=False)


@pytest.mark.parametrize("dim,group", [(64, 4), (128, 2), (256, 2)])
def test_long_tails_and_prompts(dim, group):
    """Tails longer than the prefix; a prompt chunk behind it next to single tokens."""
    run([5, dim], [1, 300, 1], [900, 420, 33], [3], [8], dim, 32, 1, group, own_columns=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q", [1, 20])
def test_tails_split_over_workgroups(dim, q):
    """Tails long enough to be dealt in parts: few rows and many."""
    run([21, dim, q], [q, q, 1], [5000, 300, 4200], [2], [20], dim, 32, 1, 16 if q > 1 else 3, own_columns=False)


@pytest.mark.parametrize("dim,q", [(64, 1), (128, 1), (256, 1), (64, 40), (128, 20), (256, 12)])
def test_many_parts_and_split_tails(dim, q):
    """A prefix in more parts than are joined at once, tails in parts, few rows and many."""
    run([23, dim, q], [q, 1], [4500, 40], [2], [110], dim, 32, 1, 16 if q > 1 else 3, own_columns=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_several_row_tiles(dim):
    """Requests of more rows than a workgroup takes of them, over a prefix in parts."""
    run([22, dim], [9, 1, 7], [30, 1, 12], [3], [64], dim, 32, 2, 8, own_columns=False)


def test_queries_inside_the_prefix():
    """A request whose queries do not all stand behind the shared pages reads its own row."""
    run(6, [1, 4, 40, 1], [9, 20, 50, 7], [4], [4], 64, 16, 2, 2, inside=[(1, 66), (2, 40), (3, 0)])
    run(7, [1, 1], [1, 1], [2], [4], 128, 16, 1, 2, inside=[(1, 64)])  # the token is the prefix's last


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_holes(dim):
    """Entries that are no page of the cache are not visible, in the prefix or behind it; all of them gone gives zeros."""
    bad = [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1]
    run([8, dim], [2, 1], [40, 20], [2], [3], dim, 16, 2, 2, holes=[("prefix", 0, 1, bad[0]), ("own", 0, 3, bad[1])])
    args, got = run([9, dim], [1, 1], [16, 16], [2], [2], dim, 16, 1, 2,
                    holes=[("prefix", 0, 0, bad[2]), ("prefix", 0, 1, bad[3]), ("own", 1, 2, -1)])
    assert np.abs(got[0]).max() > 0 and (got[1] == 0).all()
    run([10, dim], [1] * 80, [5] * 80, [80], [2], dim, 16, 1, 4, holes=[("prefix", 0, 1, -1)])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_bounds(dim):
    """A group of more pages than max_shared shares the first of them; keys past max_kv are left out."""
    run([11, dim], [1, 1], [50, 9], [2], [9], dim, 16, 1, 3, max_shared=4, spoil=False)
    run([12, dim], [1, 1], [50, 9], [2], [4], dim, 16, 1, 3, max_kv=90, spoil=False)
    run([13, dim], [1, 1], [50, 9], [2], [4], dim, 16, 1, 3, max_kv=40, spoil=False)


@pytest.mark.parametrize("dim,page,heads,group", SHAPES)
def test_wild_scales_and_sharp_scores(dim, page, heads, group):
    run([14, dim], [1, 2], [60, 40], [2], [max(1, 400 // page)], dim, page, heads, group, wild=True)
    run([15, dim], [1, 2], [60, 40], [2], [max(1, 400 // page)], dim, page, heads, group, sharp=12.0)
    run([16, dim], [1, 2], [60, 40], [2], [max(1, 400 // page)], dim, page, heads, group, scale=-0.4)
    run([17, dim], [1, 2], [60, 40], [2], [max(1, 400 // page)], dim, page, heads, group, scale=0.0)


def test_many_requests_and_groups():
    """More than 64 requests and groups, which the workgroups sum together."""
    g = np.random.default_rng(18)
    run(18, [1] * 300, [int(t) for t in g.integers(1, 40, 300)], [3] * 90, [int(p) for p in g.integers(0, 6, 90)], 64, 16, 1,
        2, g0=7, own_columns=False)


def test_offsets_out_of_order_stay_inside():
    """Starts that decrease or lie outside name no request twice and none outside; the others keep their results."""
    args, got = run(19, [1] * 6, [20] * 6, [6], [3], 64, 16, 1, 2)
    for bad in ([-5, 100], [4, 2], [9, 9], [2 ** 31 - 1, -2 ** 31]):
        args[9] = i32(bad)
        args[19].fill_(0)
        B.pn_kv4_attn_shared(*args)
        sync()
        want = got if bad == [-5, 100] else None  # all six
        out = args[19][:6, :128].reshape(6, 2, 64).double().cpu().numpy()
        # else alone: over the same pages, in their own rows; each side is off by three half
        # steps of fp16 of the largest value, 8 scales of 0.12 times 5 deviations
        assert np.abs(out - got).max() <= 6 * 2.0 ** -11 * 4.8
        if want is not None:
            assert np.array_equal(out, want)


@pytest.mark.parametrize("dim,members", [(128, 5), (128, 70), (256, 70)])
def test_stream_and_graph(dim, members):
    args, got = run([20, dim], [1] * members, [30] * members, [members], [70], dim, 16, 1, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    first = args[19].clone()
    with torch.cuda.stream(side):
        B.pn_kv4_attn_shared(*args)
        side.synchronize()
        assert torch.equal(args[19], first)
        with torch.cuda.graph(graph, stream=side):
            B.pn_kv4_attn_shared(*args)
    for scale in (0.5, 2.0, 1.0):
        args[1].mul_(scale)
        B.pn_kv4_attn_shared(*args)
        sync()
        eager = args[19].clone()
        args[19].fill_(9.0)
        graph.replay()
        sync()
        assert torch.equal(args[19], eager)
