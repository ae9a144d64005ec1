"""The attention-side operators on the GPU against plain 64-bit
implementations (kv4_ref): batch plans, norm + rotation + store into the
pn4t cache, attention over it, draft verification."""
import numpy as np
import pytest

import kv4_ref as R
from gpu_util import dev, say, sync

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_quantized_decode_pn3t_amd import _binding as B  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield


def i32(a):
    return dev(np.asarray(a, np.int32))


# ---- plan -----------------------------------------------------------------
def run_plan(ctx, new, held, free, page, table, max_pages, max_tokens):
    n = len(ctx)
    t = i32(table)
    o = dict(held_out=i32([7] * n), q_start=i32([7] * (n + 1)), kv_len=i32([7] * n), positions=i32([7] * max_tokens),
             info=i32([7, 7]))
    slots = dev(np.full(max_tokens, 7, np.int64))
    f = i32(free) if len(free) else None
    B.pn_kv4_plan(i32(ctx), i32(new), i32(held), n, f, len(free), page, t, t.shape[1], max_pages, o["held_out"],
                  o["q_start"], o["kv_len"], o["positions"], slots, max_tokens, o["info"])
    sync()
    assert B.pn_variant_name(B.pn_last_variant()) == "kv4_plan"
    got = {k: v.cpu().numpy() for k, v in o.items()}
    return dict(got, table=t.cpu().numpy(), slots=slots.cpu().numpy())


def check_plan(args):
    got, want = run_plan(*args), R.plan(*args)
    for k in want:
        assert np.array_equal(got[k], np.asarray(want[k])), (k, got[k], want[k])


@pytest.mark.parametrize("n", [1, 2, 63, 1000, 1025, 8192])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_plan_ragged(n, page):
    g = np.random.default_rng([n, page])
    ctx, new = g.integers(0, 700, n), g.integers(0, 9, n)
    new[g.random(n) < 0.2] = 0
    ctx[g.random(n) < 0.2] = 0
    if n < 2000:
        new[0] = 300
    held = -(-ctx // page) + (g.random(n) < 0.2)
    width = (1100 + page - 1) // page + 2
    pool = g.permutation(n * width)
    table = np.full((n, width + 3), -5)  # ld_table past max_pages
    at = 0
    for b in range(n):
        table[b, :held[b]] = pool[at:at + held[b]]
        at += held[b]
    need = np.maximum(0, -(-(ctx + new) // page) - held).sum()
    say("plan n=%d page=%d fresh=%d tokens=%d" % (n, page, need, new.sum()))
    check_plan((ctx, new, held, pool[at:at + need + 2], page, table, width, int(new.sum()) + 70))


def test_plan_shortages():
    """Free pages that run out, narrow tables, tokens past max_tokens, negative lengths, nothing new."""
    ctx, new, held = [10, 0, 33, 5, -3, 20], [30, 40, 0, 3, 17, -1], [1, 0, 3, 1, 0, 2]
    table = np.full((6, 4), -1)
    table[0, 0], table[2, :3], table[3, 0], table[5, :2] = 9, [8, 7, 6], 5, [4, 3]
    for free in ([20, 21, 22, 23, 24, 25, 26], [20, 21, 22], [20], []):
        for width in (4, 2, 1):
            for tokens in (200, 45, 1):
                check_plan((ctx, new, held, free, 16, table, width, tokens))
    check_plan(([5], [0], [1], [], 16, [[3]], 1, 4))
    check_plan(([0], [1], [0], [3], 16, [[-1]], 1, 1))


def test_plan_saturates():
    """Lengths whose sums pass 2^31: nothing wraps, in-range tokens stay right."""
    big = 2 ** 31 - 1
    got = run_plan([3, big], [big, big], [1, 0], [8], 16, [[5, -1], [-1, -1]], 2, 40)
    assert got["q_start"].tolist() == [0, big, big]
    assert got["kv_len"].tolist() == [big, big]
    assert got["positions"].tolist() == list(range(3, 43))
    want = [5 * 16 + p if p < 16 else 8 * 16 + p - 16 if p < 32 else -1 for p in range(3, 43)]
    assert got["slots"].tolist() == want
    assert got["info"].tolist() == [1, big]


# ---- store and load ---------------------------------------------------------
def run_store(seed, T, dim, page, kv_heads, group, half, rot, pairs, norm=True, far=5000, bad=False, eps=1e-6):
    g = np.random.default_rng(seed)
    q_heads = kv_heads * group
    kind = np.float16 if half else np.float32
    unit = 8 if half else 4
    rows, ld = [], []
    for h in (q_heads, kv_heads, kv_heads):
        pad = int(g.integers(0, 3)) * unit
        rows.append((g.standard_normal((T, h * dim + pad)) * np.exp(g.standard_normal((T, 1)))).astype(kind))
        ld.append(h * dim + pad)
    num_pages = T // page + 4
    slots = g.permutation(num_pages * page)[:T].astype(np.int64)
    positions = g.integers(0, far, T)
    if bad:
        slots[1::5] = -1
        slots[2::5] = num_pages * page + g.integers(0, 100, len(slots[2::5]))
        positions[3::5] = -1
    gains = [1 + 0.3 * g.standard_normal(dim).astype(np.float32) if norm else None for _ in range(2)]
    inv = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    before = g.integers(0, 256, (num_pages, R.page_bytes(page, kv_heads, dim))).astype(np.uint8)
    pages = dev(before)
    ldo = q_heads * dim + 8
    q_out = torch.full((T, ldo), 9.0, dtype=torch.float16, device="cuda")
    cache = B.KV4Cache(pages, num_pages, page, kv_heads, dim)
    d = [dev(r) for r in rows]
    gd = [dev(x.astype(np.float32)) if norm else None for x in gains]
    sl = dev(slots)
    B.pn_kv4_store(cache, T, d[0], d[1], d[2], "f16" if half else "f32", ld[0], ld[1], ld[2], q_heads, gd[0], gd[1],
                   eps, dev(inv) if rot else None, rot, pairs, i32(positions), sl, q_out, ldo)
    sync()
    assert B.pn_variant_name(B.pn_last_variant()) == "kv4_store"
    # expected
    x = [r[:, :h * dim] for r, h in zip(rows, (q_heads, kv_heads, kv_heads))]
    ok = positions >= 0
    there = ok & (slots >= 0) & (slots < num_pages * page)
    q, k = R.store(x[:2], (q_heads, kv_heads), gains, eps, inv, rot, pairs, np.maximum(positions, 0), dim)
    v = x[2].astype(np.float64).reshape(T, kv_heads, dim)
    # queries: fp32 through norm (sum of dim squares, root, division, two products) and rotation, then fp16
    got = q_out.cpu().numpy()
    assert np.all(got[:, q_heads * dim:] == 9) and np.all(got[~ok] == 9)
    near = np.abs(q)
    if rot:
        a, b = (near[..., 0:rot:2], near[..., 1:rot:2]) if pairs else (near[..., :rot // 2], near[..., rot // 2:rot])
        both = a + b
        both = np.repeat(both, 2, -1) if pairs else np.concatenate((both, both), -1)
        # a turn keeps the length, so |a| + |b| before it is at most sqrt 2 of that after it
        near = np.concatenate((1.5 * both, near[..., rot:]), -1)
    tol = 2.0 ** -11 * np.abs(q) + (dim / 8 + 24) * 2.0 ** -24 * near + 2.0 ** -25
    err = np.abs(got[:, :q_heads * dim].reshape(q.shape).astype(np.float64) - q)
    assert np.all(err[ok] <= tol[ok]), float((err[ok] / tol[ok]).max())
    # the cache, byte for byte: places of other tokens keep what they held
    want = before.copy()
    for t in np.nonzero(there)[0]:
        R.put(want, page, kv_heads, dim, slots[t], "k", *R.quantize(k[t]))
        R.put(want, page, kv_heads, dim, slots[t], "v", *R.quantize(v[t]))
    after = pages.cpu().numpy()
    assert np.array_equal(after, want), int((after != want).sum())
    # and back
    ko = torch.full((T, kv_heads * dim), 9.0, device="cuda")
    vo = torch.full((T, kv_heads * dim), 9.0, device="cuda")
    B.pn_kv4_load(cache, sl, T, ko, vo)
    sync()
    inside = (slots >= 0) & (slots < num_pages * page)
    kr, vr = R.get(want, page, kv_heads, dim, np.where(inside, slots, 0))
    kr[~inside], vr[~inside] = 0, 0
    fine = np.isfinite(kr).reshape(T, -1) & np.isfinite(vr).reshape(T, -1)
    for o, r in ((ko, kr), (vo, vr)):
        o = o.cpu().numpy()
        assert np.array_equal(o[fine], r.reshape(T, -1).astype(np.float32)[fine])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,page,kv_heads,group,part", [(1, 16, 1, 1, 1), (7, 32, 4, 6, 2), (37, 64, 3, 5, 4),
                                                        (70, 256, 2, 8, 1)])
def test_store(dim, half, pairs, T, page, kv_heads, group, part):
    rot = dim // part
    say("store dim=%d half=%s pairs=%s T=%d rot=%d" % (dim, half, pairs, T, rot))
    run_store([dim, half, pairs, T], T, dim, page, kv_heads, group, half, rot, pairs)


def test_store_bad_places_and_padding():
    for dim in (64, 128, 256):
        run_store([5, dim], 43, dim, 16, 2, 3, False, 32, False, bad=True)


def test_store_without_norm_or_rotation():
    run_store(6, 9, 128, 16, 2, 3, False, 0, False, norm=False)
    run_store(7, 9, 128, 16, 2, 3, True, 48, False, norm=False)
    run_store(8, 9, 128, 16, 2, 3, True, 112, True, eps=0.5)


def test_store_far_positions():
    run_store(9, 33, 128, 64, 2, 2, False, 128, False, far=2 ** 31 - 1)


def test_store_many_tokens():
    run_store(10, 700, 64, 64, 1, 2, False, 64, False)


def values_row(v, T, heads, dim, page=16):
    """Store v [T, heads, dim] fp32 as keys and values (no norm, no rotation); returns the pages."""
    num_pages = T // page + 1
    pages = torch.zeros(num_pages, R.page_bytes(page, heads, dim), dtype=torch.uint8, device="cuda")
    cache = B.KV4Cache(pages, num_pages, page, heads, dim)
    x = dev(v.reshape(T, -1))
    slots = dev(np.arange(T, dtype=np.int64))
    B.pn_kv4_store(cache, T, None, x, x, "f32", 0, heads * dim, heads * dim, 0, None, None, 0.0, None, 0, False,
                   i32(np.zeros(T)), slots, None, 0)
    sync()
    return pages.cpu().numpy()


def test_store_special_values():
    """Zero blocks, scales that underflow or saturate, equal magnitudes, ties, infinities and NaN."""
    g = np.random.default_rng(3)
    T, dim = 12, 64
    v = g.standard_normal((T, 1, dim)).astype(np.float32)
    v[0] = 0
    v[1] *= 1e-9
    v[2] = v[2] * np.float32(2e-7)
    v[3, 0, 7], v[3, 0, 11] = -9, 9
    v[4, 0] = np.arange(-32, 32) / 4
    v[5] *= 1e6
    v[6, 0, 3] = np.inf
    v[7, 0, 3] = -np.inf
    v[8, 0, 5] = np.nan
    v[9] = np.nan
    v[10] = -0.0
    v[11] = 3e38
    want = np.zeros((1, R.page_bytes(16, 1, dim)), np.uint8)
    for t in range(T):
        for side in "kv":
            R.put(want, 16, 1, dim, t, side, *R.quantize(v[t]))
    assert np.array_equal(values_row(v, T, 1, dim), want)


def test_store_matches_the_c_oracle():
    g = np.random.default_rng(4)
    v = (g.standard_normal((50, 2, 128)) * np.exp(2 * g.standard_normal((50, 2, 1)))).astype(np.float32)
    d, n = R.pnref_codes(v.reshape(100, 128))
    want = np.zeros((4, R.page_bytes(16, 2, 128)), np.uint8)
    for t in range(50):
        for side in "kv":
            R.put(want, 16, 2, 128, t, side, d.reshape(50, 2, -1)[t], n.reshape(50, 2, -1)[t])
    assert np.array_equal(values_row(v, 50, 2, 128), want)


# ---- attention ---------------------------------------------------------------
def make_cache(g, num_pages, page, heads, dim, wild=False):
    """Random codes and scales in every place (fast: no quantizer)."""
    pages = g.integers(0, 256, (num_pages, R.page_bytes(page, heads, dim))).astype(np.uint8)
    r = dim // 64
    per = page * (dim + dim // 16)
    v = pages.reshape(num_pages, heads, per)
    sc = (g.standard_normal((num_pages, heads, 2, page * r)) * 0.12).astype(np.float16)
    if wild:  # value scales over many sizes, and zeros
        sc[:, :, 1] = (sc[:, :, 1].astype(np.float32) * 2.0 ** g.integers(-12, 13, sc[:, :, 1].shape)).astype(np.float16)
        sc[:, :, 1, ::7] = 0
    v[:, :, page * dim:] = sc.reshape(num_pages, heads, -1).view(np.uint8)
    return pages


def run_attn(seed, q_lens, kv_lens, dim, page, heads, group, window=0, sinks=0, ws_mb=64, wild=False, scale=None,
             spoil=True, holes=(), max_q=None, max_kv=None, sharp=1.0):
    g = np.random.default_rng(seed)
    n, q_heads = len(q_lens), heads * group
    q_start = np.concatenate(([0], np.cumsum(q_lens)))
    T = int(q_start[-1])
    top = max(max(kv_lens), 1) if max_kv is None else max_kv
    width = -(-top // page)
    used = [-(-max(k, 0) // page) for k in kv_lens]
    num_pages = sum(used) + 2
    pages = make_cache(g, num_pages, page, heads, dim, wild)
    ids = g.permutation(num_pages)
    table = np.full((n, width + 2), -1)
    at = 0
    for b in range(n):
        table[b, :used[b]] = ids[at:at + used[b]]
        at += used[b]
    if spoil:  # what was never written holds NaN and infinite scales
        r = dim // 64
        for b in range(n):
            for t in range(kv_lens[b], used[b] * page):
                for h in range(heads):
                    base = h * page * (dim + dim // 16) + page * dim
                    for side in (0, 2 * page * r):
                        o = base + side + 2 * r * (t % page)
                        pages[table[b, t // page], o:o + 2 * r] = np.tile([0x00, 0x7e if t % 2 else 0xfc], r)
    for b, c, entry in holes:
        table[b, c] = entry
    scale = dim ** -0.5 if scale is None else scale
    ld = q_heads * dim + 8
    q = (g.standard_normal((T, ld)) * sharp).astype(np.float16)
    out = torch.full((T, ld), 9.0, dtype=torch.float16, device="cuda")
    cache = B.KV4Cache(dev(pages), num_pages, page, heads, dim)
    ws = torch.full((ws_mb << 18,), float("nan"), device="cuda") if ws_mb else None
    args = (cache, dev(q), ld, q_heads, i32(q_start), i32(kv_lens), i32(table), width + 2, n, T,
            max_q or max(max(q_lens), 1), top, scale, window, sinks, out, ld, ws, ws_mb << 20)
    B.pn_kv4_attn(*args)
    sync()
    got = out.cpu().numpy()
    again = torch.full((T, ld), 9.0, dtype=torch.float16, device="cuda")
    B.pn_kv4_attn(*args[:15], again, *args[16:])
    sync()
    assert np.array_equal(got.view(np.uint16), again.cpu().numpy().view(np.uint16)), "two runs differ"
    want, bound = R.attend(q[:, :q_heads * dim].reshape(T, q_heads, dim), pages, page, heads, dim, q_start, kv_lens,
                           table, np.float64(np.float32(scale)), window, sinks, num_pages)
    if max_kv is not None or max_q is not None:
        return got, want, bound
    assert np.all(got[:, q_heads * dim:] == 9)
    got = got[:, :q_heads * dim].reshape(want.shape).astype(np.float64)
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0].tolist(), got[bad][:4], want[bad][:4], bound[bad][:4])


SHAPES = [(64, 16, 2, 1), (64, 64, 1, 16), (128, 16, 2, 6), (128, 256, 1, 3), (256, 32, 1, 6), (256, 16, 3, 2)]


@pytest.mark.parametrize("dim,page,heads,group", SHAPES)
@pytest.mark.parametrize("kv", [1, 2, 15, 16, 17, 31, 32, 33, 64, 100, 257])
def test_attn_single_token_lengths(dim, page, heads, group, kv):
    say("attn dim=%d page=%d heads=%d group=%d kv=%d" % (dim, page, heads, group, kv))
    run_attn([dim, kv], [1], [kv], dim, page, heads, group)


@pytest.mark.parametrize("dim,page,heads,group", SHAPES)
def test_attn_ragged_tokens(dim, page, heads, group):
    say("attn ragged dim=%d page=%d" % (dim, page))
    run_attn([1, dim], [1] * 9, [5, 700, 1, 64, 33, 1500, 2, 129, 16], dim, page, heads, group)


@pytest.mark.parametrize("dim,page,heads,group", SHAPES)
@pytest.mark.parametrize("q", [2, 5, 8, 16])
def test_attn_drafts(dim, page, heads, group, q):
    say("attn drafts dim=%d page=%d q=%d" % (dim, page, q))
    run_attn([2, dim, q], [q, 1, q], [q, 300, 77 + q], dim, page, heads, group)


@pytest.mark.parametrize("dim,page,heads,group", SHAPES)
@pytest.mark.parametrize("q,kv", [(40, 40), (130, 130), (97, 331)])
def test_attn_prompts(dim, page, heads, group, q, kv):
    say("attn prompt dim=%d page=%d q=%d kv=%d" % (dim, page, q, kv))
    run_attn([3, dim, q], [q, 3, q - 20], [kv, 50, q - 20], dim, page, heads, group)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (32, 0), (33, 40), (100, 4), (64, 16), (1000, 4)])
@pytest.mark.parametrize("dim,page,heads,group", [(64, 16, 1, 3), (128, 64, 2, 2), (256, 16, 1, 6)])
def test_attn_window(dim, page, heads, group, window, sinks):
    say("attn window=%d sinks=%d dim=%d" % (window, sinks, dim))
    run_attn([4, dim, window], [1, 8, 90, 1], [700, 400, 333, 3], dim, page, heads, group, window, sinks)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attn_long(dim):
    """Many splits, one row; and a workspace that holds none, or only some, of them."""
    for mb in (64, 0, 1):
        say("attn long dim=%d ws=%d MB" % (dim, mb))
        run_attn([5, dim], [1, 1], [9000, 4100], dim, 64, 2, 4, ws_mb=mb)


def test_attn_empty():
    """No queries, no keys, more queries than keys (the first ones see nothing), lengths below zero."""
    run_attn(6, [0, 1, 0, 3, 5, 1], [5, 0, 0, 7, 2, -4], 128, 16, 2, 3)
    run_attn(7, [1], [0], 64, 16, 1, 1)
    run_attn(8, [70], [9], 64, 16, 1, 4)


def test_attn_holes():
    """Pages that are not of the cache: their tokens are not visible; a row may lose all its keys."""
    run_attn(9, [1, 4, 1], [100, 90, 20], 128, 16, 2, 3, holes=((0, 2, -1), (0, 6, 10 ** 6), (1, 0, -7), (2, 0, -1),
                                                               (2, 1, 2 ** 31 - 1)))
    run_attn(10, [60, 1], [200, 64], 64, 64, 1, 4, holes=((0, 1, -1), (1, 0, -1)))


@pytest.mark.parametrize("dim,page,heads,group", SHAPES)
def test_attn_wild_scales(dim, page, heads, group):
    """Value scales from 2^-16 to 2^9 and zeros side by side: nothing overflows, the small ones count."""
    run_attn([11, dim], [1, 8, 40], [500, 300, 99], dim, page, heads, group, wild=True)


def test_attn_sharp_scores():
    """Scores hundreds apart: one key takes all, wherever it is."""
    run_attn(12, [1, 20], [1000, 200], 128, 16, 1, 4, sharp=40.0)
    run_attn(13, [1, 20], [1000, 200], 128, 16, 1, 4, scale=-0.5)
    run_attn(14, [1, 20], [1000, 200], 128, 16, 1, 4, scale=0.0)


def test_attn_bounds_left_out():
    """Queries past max_q are left alone; keys past max_kv are left out without a fault."""
    got, want, bound = run_attn(15, [9, 4], [60, 50], 64, 16, 1, 2, max_q=5)
    got = got[:, :128].reshape(want.shape).astype(np.float64)
    for t in list(range(5)) + list(range(9, 13)):
        assert np.all(np.abs(got[t] - want[t]) <= bound[t])
    assert np.all(got[5:9] == 9)
    run_attn(16, [1, 1], [60, 50], 64, 16, 1, 2, max_kv=40)


def test_attn_other_stream_and_graph():
    """Plan, store, attention and verification captured together, replayed between eager calls."""
    g = np.random.default_rng(17)
    n, dim, page, heads, group = 5, 128, 16, 2, 3
    q_heads, T = heads * group, 5 * 3
    ctx, held = np.array([40, 0, 17, 100, 3]), np.array([3, 0, 2, 7, 1])
    num_pages, width = 60, 12
    pages = dev(make_cache(g, num_pages, page, heads, dim))
    cache = B.KV4Cache(pages, num_pages, page, heads, dim)
    pool = g.permutation(num_pages)
    table = np.full((n, width), -1)
    at = 0
    for b in range(n):
        table[b, :held[b]] = pool[at:at + held[b]]
        at += held[b]
    table, free = i32(table), i32(pool[at:])
    ctx_d, new_d, held_d = i32(ctx), i32([3] * n), i32(held)
    outs = [torch.empty(n + 1, dtype=torch.int32, device="cuda") for _ in range(5)]
    held_out, q_start, kv_len, info, acc = outs
    positions, slots = i32(np.zeros(T)), dev(np.zeros(T, np.int64))
    x = dev(g.standard_normal((T, (q_heads + 2 * heads) * dim)).astype(np.float32))
    ld = x.shape[1]
    gain = dev(np.ones(dim, np.float32))
    inv = dev((10000.0 ** (-np.arange(dim // 2) / (dim // 2))).astype(np.float32))
    q = torch.empty(T, q_heads * dim, dtype=torch.float16, device="cuda")
    o = torch.empty_like(q)
    V, k = 5000, 2
    p = torch.softmax(2 * torch.randn(n, k + 1, V, device="cuda"), -1)
    d = torch.softmax(2 * torch.randn(n, k, V, device="cuda"), -1)
    toks, u = d.argmax(-1).int(), torch.rand(n, k + 1, device="cuda")
    out = torch.empty(n, k + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def step():
        B.pn_kv4_plan(ctx_d, new_d, held_d, n, free, free.numel(), page, table, width, width, held_out, q_start, kv_len,
                      positions, slots, T, info)
        B.pn_kv4_store(cache, T, x, x[:, q_heads * dim:], x[:, (q_heads + heads) * dim:], "f32", ld, ld, ld, q_heads,
                       gain, gain, 1e-6, inv, dim, False, positions, slots, q, q_heads * dim)
        B.pn_kv4_attn(cache, q, q_heads * dim, q_heads, q_start, kv_len, table, width, n, T, 3, width * page,
                      dim ** -0.5, 0, 0, o, q_heads * dim, ws, ws.numel())
        B.pn_spec_verify(p, V, d, V, toks, k, None, u, k + 1, n, k, V, out, k + 1, acc, ws, ws.numel())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    first = [t.clone() for t in (o, out, pages, table)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for scale in (1.0, 0.5, 2.0, 1.0):
        x.mul_(scale)
        step()
        sync()
        eager = [t.clone() for t in (o, out, pages, table)]
        o.zero_(), out.zero_()
        graph.replay()
        sync()
        for a, b in zip(eager, (o, out, pages, table)):
            assert torch.equal(a, b)
    for a, b in zip(first, eager):
        assert torch.equal(a, b)


# ---- draft verification --------------------------------------------------------
def run_verify(target, draft, tokens, n_draft, u, pad=0):
    n, k1, V = target.shape
    k = k1 - 1
    t = torch.full((n, k1, V + pad), 0.25, device="cuda")
    t[..., :V] = dev(target)
    d = None
    if draft is not None:
        d = torch.full((n, k, V + pad), 0.25, device="cuda")
        d[..., :V] = dev(draft)
    out = torch.full((n, k1 + 1), 77, dtype=torch.int32, device="cuda")
    acc = torch.full((n,), 77, dtype=torch.int32, device="cuda")
    size = B.pn_spec_workspace(n, V)
    ws = torch.full((size + 64,), 0xff, dtype=torch.uint8, device="cuda")
    tok = i32(np.concatenate((tokens, np.full((n, 2), 10 ** 9)), 1))
    B.pn_spec_verify(t, V + pad, d, V + pad, tok, k + 2, None if n_draft is None else i32(n_draft), dev(u), k1, n, k, V,
                     out, k1 + 1, acc, ws, size)
    sync()
    assert B.pn_variant_name(B.pn_last_variant()) == "spec_verify"
    assert bool((ws[size:] == 0xff).all()) and bool((out[:, k1] == 77).all())
    return out.cpu().numpy()[:, :k1], acc.cpu().numpy()


def dyadic(g, shape, bits=20):
    """Entries that are multiples of 2^-20: every sum is exact."""
    x = g.integers(0, 2 ** 10, shape) * (g.random(shape) < 0.3)
    return (x * 2.0 ** -bits).astype(np.float32)


@pytest.mark.parametrize("V", [1, 2, 63, 1000, 4095, 4096, 4097, 70001])
@pytest.mark.parametrize("k", [0, 1, 3, 7])
@pytest.mark.parametrize("probs", [True, False])
def test_verify(V, k, probs):
    g = np.random.default_rng([V, k, probs])
    n = 9
    say("verify V=%d k=%d probs=%s" % (V, k, probs))
    target = dyadic(g, (n, k + 1, V))
    draft = dyadic(g, (n, k, V)) if probs else None
    if probs:
        same = g.random((n, k, 1)) < 0.5  # rows whose drafts are mostly accepted
        draft = np.where(same, target[:, :k] * 0.5, draft).astype(np.float32)
    tokens = g.integers(0, V, (n, k))
    u = g.random((n, k + 1)).astype(np.float32)
    u[:, :k] *= 2.0 ** -g.integers(0, 12, (n, k)).astype(np.float32)
    for n_draft in (None, g.integers(-1, k + 3, n)):
        got = run_verify(target, draft, tokens, n_draft, u, pad=3)
        want = R.verify(target, draft, tokens, n_draft, u)
        assert np.array_equal(got[1], want[1]), (got[1], want[1])
        assert np.array_equal(got[0], want[0]), (got[0], want[0])


def test_verify_borders():
    """u exactly on a prefix sum, and exactly on the acceptance ratio."""
    V, n = 9000, 64
    g = np.random.default_rng(1)
    target = np.zeros((n, 2, V), np.float32)
    spots = np.sort(g.permutation(V)[:1024])
    target[:, :, spots] = 2.0 ** -10  # sums to 1
    draft = np.zeros((n, 1, V), np.float32)
    draft[:, 0, spots[:512]] = 2.0 ** -9
    tokens = np.full((n, 1), spots[3])
    u = np.zeros((n, 2), np.float32)
    u[:, 0] = np.where(np.arange(n) % 2, 0.5, np.nextafter(np.float32(0.5), np.float32(0)))  # p / q = 1/2: refused at it
    u[:, 1] = np.arange(n) * 16 / 1024
    got = run_verify(target, draft, tokens, None, u)
    want = R.verify(target, draft, tokens, None, u)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert want[1].tolist() == [1 - i % 2 for i in range(n)]


def test_verify_degenerate():
    """Nothing left of p - q, empty rows, entries that do not count, tokens out of range, u at 0 and at 1."""
    V = 5000
    target = np.zeros((8, 2, V), np.float32)
    draft = np.zeros((8, 1, V), np.float32)
    tokens = np.full((8, 1), 7)
    u = np.full((8, 2), 0.5, np.float32)
    target[0, 0, 7], draft[0, 0, 7] = 0.25, 1.0  # refused, p - q empty: from p
    target[1] = 0  # nothing at all: -1
    target[2, 0, [3, 4500]] = [np.nan, 0.5]
    target[2, 0, 9] = np.inf
    draft[2, 0, 7] = 1
    target[3, 0, [10, 4999]] = 0.5
    tokens[3] = V
    target[4, 0, [10, 4999]] = 0.5
    tokens[4] = -1
    target[5, 0, 7], draft[5, 0, 7] = 1.0, 0.5
    target[5, 1, [11, 12]] = 0.5
    u[5, 1] = 0.0
    target[6] = target[5]
    draft[6] = draft[5]
    u[6, 1] = 1.0  # past every prefix: the last entry that counts
    target[7, 0, [1, 2, 3]] = [-1.0, 0.5, -0.5]
    draft[7, 0, 7] = 1
    for d in (draft, None):
        got, want = run_verify(target, d, tokens, None, u), R.verify(target, d, tokens, None, u)
        assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0]), (got, want)


# ---- places past 32 bits ----------------------------------------------------
@pytest.mark.parametrize("dim,q", [(64, 1), (128, 5), (256, 1), (128, 300)])
def test_far_pages_and_rows(dim, q):
    """A cache of over 5 GiB, used at its far end, and query rows over
    6 GiB give what a small cache and dense rows give."""
    heads, group, page, n = 2, 3, 64, 2
    q_heads, kv = heads * group, 333
    per = B.pn_kv4_page_bytes(page, heads, dim)
    width = -(-kv // page)
    num = (5 << 30) // per + n * width
    g = torch.Generator(device="cuda")
    g.manual_seed(dim + q)
    k, v = (torch.randn((n * kv, heads * dim), generator=g, device="cuda") for _ in range(2))
    rows = torch.randn((n * q, q_heads * dim), generator=g, device="cuda").half()
    pos = torch.arange(kv, device="cuda").repeat(n)
    outs, loads = [], []
    far = (3 << 30) // (8 * (n * q - 1)) * 8  # the last row is 6 GiB on
    for count, first, ld in ((n * width, 0, q_heads * dim), (num, num - n * width, far)):
        say("far: dim=%d q=%d pages=%d ld=%d" % (dim, q, count, ld))
        pages = torch.empty(count * per, dtype=torch.uint8, device="cuda")
        cache = B.KV4Cache(pages, count, page, heads, dim)
        table = (torch.arange(n * width, device="cuda") + first).int().view(n, width)
        slots = table.long().repeat_interleave(page, 1)[:, :kv].reshape(-1) * page + pos % page
        B.pn_kv4_store(cache, n * kv, None, k, v, "f32", 0, heads * dim, heads * dim, q_heads, None, None, 0.0, None,
                       0, False, pos.int(), slots, None, 0)
        back = torch.empty((2, n * kv, heads * dim), device="cuda")
        B.pn_kv4_load(cache, slots, n * kv, back[0], back[1])
        loads.append(back)
        flat = torch.empty((n * q - 1) * ld + q_heads * dim, dtype=torch.float16, device="cuda")
        at = flat.as_strided(rows.shape, (ld, 1))
        at.copy_(rows)
        out = torch.empty_like(flat)
        need = B.pn_kv4_attn_workspace(cache, q_heads, n, n * q, q, kv)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        B.pn_kv4_attn(cache, flat, ld, q_heads, i32([0, q, 2 * q]), i32([kv, kv - 20]), table, width, n, n * q, q, kv,
                      dim ** -0.5, 0, 0, out, ld, ws, need)
        sync()
        outs.append(out.as_strided(rows.shape, (ld, 1)).clone())
    assert torch.equal(loads[0], loads[1])
    assert outs[0].isfinite().all() and outs[0].abs().max() > 0
    assert torch.equal(outs[0], outs[1])
