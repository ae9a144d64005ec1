"""Edges of the attention-side operators on the GPU, against plain 64-bit
implementations: small values, windows wider than any context, batches above
64 requests, items cut between workgroups in every kernel, workspaces of every
size, missing pages, bounds of lengths."""
import numpy as np
import pytest

import kv4_ref as R
from gpu_util import dev, say, sync
from test_gpu_kv4 import i32, make_cache

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from bit_quantized_decode_pn3t_amd import _binding as B  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield


def attend(q, pages, page, heads, dim, q_start, kv_len, table, scale, window, sinks, num_pages, max_kv):
    """kv4_ref.attend, a request's rows at once and keys past max_kv left out: (out, bound)."""
    group = q.shape[1] // heads
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(len(kv_len)):
        n, q0, q1 = max(0, int(kv_len[b])), int(q_start[b]), int(q_start[b + 1])
        keys = min(n, max_kv)
        if q1 <= q0 or keys == 0:
            continue
        t = np.arange(keys)
        entry = np.asarray(table[b])[np.minimum(t // page, table.shape[1] - 1)]
        there = (entry >= 0) & (entry < num_pages)
        k, v = R.get(pages, page, heads, dim, np.where(there, entry, 0).astype(np.int64) * page + t % page)
        p = n - (q1 - q0) + np.arange(q1 - q0)[:, None]
        see = there & (t <= p)
        if window > 0:
            see &= (t > p - window) | (t < sinks)
        any_ = see.any(0)  # keys that no row sees may hold anything
        k, v = np.where(any_[:, None, None], k, 0), np.where(any_[:, None, None], v, 0)
        some = see.any(1)
        count = see.sum(1)[:, None]
        for h in range(heads):
            kk, vv = k[:, h], v[:, h]
            for i in range(h * group, (h + 1) * group):
                x = q[q0:q1, i].astype(np.float64)
                s = np.where(see, x @ kk.T * scale, -np.inf)
                mag = np.where(see, np.abs(x) @ np.abs(kk).T * abs(scale), 0).max(1)[:, None]
                w = np.exp(s - np.where(some, s.max(1), 0)[:, None])
                sum_ = np.where(some, w.sum(1), 1)[:, None]
                y, a = w @ vv / sum_, w @ np.abs(vv) / sum_
                top = np.where(see, np.abs(vv).max(1), 0).max(1)[:, None]
                eta = 2 * ((dim + 8) * 2.0 ** -24 * mag + 8 * 2.0 ** -24)
                e = a * (2 * 2.0 ** -11 + 2 * eta + (count + 64) * 2.0 ** -24) + count * top * 2.0 ** -34
                out[q0:q1, i] = y
                bound[q0:q1, i] = np.where(some[:, None], e + 2.0 ** -11 * (np.abs(y) + e) + 2.0 ** -25, 0)
    return out, bound


def run(seed, q_lens, kv_lens, dim, page, heads, group, window=0, sinks=0, share=1.0, holes=(), factor=None,
        max_q=None, max_kv=None, variant=None, scale=None, sharp=1.0):
    """One call against the plain form.  share: part of the workspace that the
    call could use; factor(b, t): what the value scales of a request's tokens
    are multiplied by; variant: the kernel that must have run."""
    g = np.random.default_rng(seed)
    n, q_heads = len(q_lens), heads * group
    q_start = np.concatenate(([0], np.cumsum(q_lens)))
    T = int(q_start[-1])
    top = max(max(kv_lens), 1) if max_kv is None else max_kv
    width = -(-max(max(kv_lens), 1) // page)
    used = [-(-max(k, 0) // page) for k in kv_lens]
    num_pages = sum(used) + 2
    pages = make_cache(g, num_pages, page, heads, dim)
    ids = g.permutation(num_pages)
    table = np.full((n, width + 2), -1)
    at, r = 0, dim // 64
    scales = pages.reshape(num_pages, heads, -1)[:, :, page * dim:].view(np.float16).reshape(num_pages, heads, 2, page, r)
    assert np.shares_memory(scales, pages)
    for b in range(n):
        table[b, :used[b]] = ids[at:at + used[b]]
        at += used[b]
        t = np.arange(used[b] * page)
        where = table[b, t // page]
        if factor is not None:
            f = np.broadcast_to(np.asarray(factor(b, t), np.float32), t.shape)
            s = scales[where, :, 1, t % page].astype(np.float32) * f[:, None, None]
            scales[where, :, 1, t % page] = s.astype(np.float16)
        past = t >= kv_lens[b]  # what was never written holds NaN and infinite scales
        scales[where[past], :, :, (t % page)[past]] = np.where(t[past] % 2, np.nan, -np.inf)[:, None, None, None]
    for b, c, entry in holes:
        table[b, c] = entry
    scale = dim ** -0.5 if scale is None else scale
    ld = q_heads * dim + 8
    q = (g.standard_normal((T, ld)) * sharp).astype(np.float16)
    cache = B.KV4Cache(dev(pages), num_pages, page, heads, dim)
    mq = max_q or max(max(q_lens), 1)
    size = int(B.pn_kv4_attn_workspace(cache, q_heads, n, T, mq, top, window, sinks) * share) // 8 * 8
    ws = torch.full((size // 4 + 64,), float("nan"), device="cuda")
    say("attn edges dim=%d page=%d heads=%dx%d q=%s kv=%s window=%d+%d ws=%d" %
        (dim, page, heads, group, q_lens[:6], kv_lens[:6], window, sinks, size))
    outs = []
    dq, ds, dl, dt = dev(q), i32(q_start), i32(kv_lens), i32(table)
    for _ in range(2):
        out = torch.full((T, ld), 9.0, dtype=torch.float16, device="cuda")
        B.pn_kv4_attn(cache, dq, ld, q_heads, ds, dl, dt, width + 2, n, T, mq, top, scale, window, sinks, out, ld,
                      ws if size else None, size)
        sync()
        outs.append(out.cpu().numpy())
    if variant:
        assert B.pn_variant_name(B.pn_last_variant()) == variant
    assert bool(ws[size // 4:].isnan().all()), "past the workspace"
    assert np.array_equal(outs[0].view(np.uint16), outs[1].view(np.uint16)), "two runs differ"
    want, bound = attend(q[:, :q_heads * dim].reshape(T, q_heads, dim), pages, page, heads, dim, q_start, kv_lens,
                         table, np.float64(np.float32(scale)), window, sinks, num_pages, top)
    got = outs[0]
    assert np.all(got[:, q_heads * dim:] == 9)
    got = got[:, :q_heads * dim].reshape(want.shape).astype(np.float64)
    ok = np.abs(got - want) <= bound
    for b in range(n):  # queries past max_q are left alone
        left = slice(q_start[b] + mq, max(q_start[b] + mq, q_start[b + 1]))
        assert np.all(got[left] == 9)
        ok[left] = True
    assert ok.all(), (int((~ok).sum()), np.argwhere(~ok)[0].tolist(), got[~ok][:4], want[~ok][:4], bound[~ok][:4])


# Single tokens, drafts (one and several 16-row groups a wave) and prompts
# (256 wide: four row groups) of each head width: (dim, page, heads, group), q.
FORMS = [((64, 16, 2, 3), 1), ((64, 16, 1, 8), 8), ((64, 64, 1, 8), 80),
         ((128, 16, 2, 3), 1), ((128, 32, 1, 6), 8), ((128, 64, 1, 6), 50),
         ((256, 64, 2, 3), 1), ((256, 32, 1, 6), 5), ((256, 16, 1, 6), 26)]


# ---- small values ---------------------------------------------------------------
@pytest.mark.parametrize("shape,q", FORMS)
@pytest.mark.parametrize("power", [-7, -10, -20])
def test_small_values(shape, q, power):
    """Value scales so small that the factor which brings them up would leave fp16."""
    run([1, -power, q], [q, 1], [300, 70], *shape, factor=lambda b, t: 2.0 ** power)


@pytest.mark.parametrize("shape,q", FORMS)
@pytest.mark.parametrize("power", [-9, -20])
def test_small_values_first(shape, q, power):
    """The first 64 tokens alone have small values, or the first 1024."""
    run([2, -power, q], [q, 1], [600, 200], *shape, factor=lambda b, t: np.where(t < 64, 2.0 ** power, 1.0))
    run([3, -power, q], [q, 1], [1300, 1100], *shape, factor=lambda b, t: np.where(t < 1024, 2.0 ** power, 1.0))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("power", [0, -6, -8, -12, -20])
def test_small_value_alone(dim, power):
    """One key with a small value."""
    run([4, dim, -power], [1, 1, 1], [1, 1, 33], dim, 16, 2, 2, factor=lambda b, t: 2.0 ** power)


# ---- windows ----------------------------------------------------------------------
@pytest.mark.parametrize("shape,q", FORMS)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 20, 2 ** 30])
def test_window_wider_than_anything(shape, q, window):
    """A window that hides nothing, with fewer keys than queries in some requests."""
    run([5, q], [q, q + 3, q], [max(1, q // 2), q + 40, 1], *shape, window=window, sinks=2)


# ---- batches above 64 requests ------------------------------------------------------
@pytest.mark.parametrize("n", [64, 65, 300, 513, 1000, 2049])
@pytest.mark.parametrize("dim,page,heads,group", [(64, 16, 2, 2), (128, 16, 1, 3), (256, 32, 1, 6)])
def test_many_requests(n, dim, page, heads, group):
    """Single tokens, drafts and a few prompts, requests without queries or
    keys among them; short ones alone, and with a few long ones that are cut."""
    g = np.random.default_rng([n, dim])
    for most, long, window, sinks in ((1, 0, 0, 0), (6, 0, 0, 0), (6, 1500, 0, 0), (6, 1500, 30, 4), (1, 2500, 700, 0)):
        q = g.integers(1, most + 1, n)
        kv = q + g.integers(0, 70, n)
        q[g.random(n) < 0.15] = 0
        kv[g.random(n) < 0.1] = 0
        if long:
            at = g.permutation(n)[:4]
            kv[at] = g.integers(long // 2, long, 4)
            q[at] = np.minimum(g.integers(1, 4 * most, 4), kv[at])
            kv[at[0]] = long
        run([6, n, dim, most], q.tolist(), kv.tolist(), dim, page, heads, group, window, sinks)


@pytest.mark.parametrize("dim,page,heads,group,q", [(64, 64, 1, 8, 70), (128, 16, 1, 6, 50), (256, 16, 1, 6, 30)])
def test_many_requests_with_prompts(dim, page, heads, group, q):
    """The kernels of many rows over more than 64 requests."""
    g = np.random.default_rng([7, dim])
    for n in (65, 140):
        lens = np.where(g.random(n) < 0.2, q, g.integers(0, 4, n))
        lens[0] = q
        kv = lens + g.integers(0, 60, n)
        kv[n // 2], lens[n // 2] = 1400, 20
        run([7, n, dim], lens.tolist(), kv.tolist(), dim, page, heads, group)


# ---- items cut between workgroups ----------------------------------------------------
# rows of the longest request: one to four 16-row groups a wave, then the kernels of many rows
ROWS = [(64, 16, 1, 5, 2), (64, 32, 1, 4, 7), (64, 16, 1, 8, 6), (64, 64, 1, 6, 11), (64, 64, 1, 8, 40),
        (64, 16, 1, 8, 65), (64, 64, 1, 16, 70),
        (128, 16, 1, 5, 2), (128, 32, 1, 4, 7), (128, 16, 1, 8, 6), (128, 64, 1, 6, 11), (128, 32, 1, 6, 42),
        (128, 16, 1, 8, 33), (128, 64, 1, 6, 90),
        (256, 16, 1, 5, 2), (256, 64, 1, 6, 8), (256, 16, 1, 6, 21), (256, 16, 1, 6, 22), (256, 32, 1, 8, 40)]


def kernel(dim, rows):
    """The kernel that takes a call whose longest request has so many rows."""
    return "kv4_prompt" if dim < 256 and rows > (512 if dim == 64 else 256) else "kv4_attn"


@pytest.mark.parametrize("share", [1.0, 0.6, 0.27, 0.1, 0.0])
@pytest.mark.parametrize("dim,page,heads,group,q", ROWS)
def test_cut_items(dim, page, heads, group, q, share):
    """More than 1024 keys: parts of items are joined, with room for all, some or none."""
    run([8, dim, q], [q, 1, q, 0], [1700, 1300, 900 + q, 40], dim, page, heads, group, share=share,
        variant=kernel(dim, q * group))


@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 3), (300, 70), (1100, 0), (5000, 4)])
@pytest.mark.parametrize("dim,page,heads,group,q", ROWS)
def test_cut_items_window(dim, page, heads, group, q, window, sinks):
    run([9, dim, q, window], [q, 1, q], [2100, 1300, 900 + q], dim, page, heads, group, window, sinks)


@pytest.mark.parametrize("dim,page,heads,group,q", ROWS)
def test_holes_and_empty_rows(dim, page, heads, group, q):
    """Pages that are not of the cache, whole requests of them, and more queries than keys."""
    last = -(-1500 // page) - 1
    holes = ((0, 0, -1), (0, 3, 10 ** 6), (0, last, -9), (1, 0, -1), (1, 1, 2 ** 31 - 1), (2, 1, -1))
    for window, sinks in ((0, 0), (60, 5)):
        run([10, dim, q, window], [q, q, q, q], [1500, min(33, 2 * page), 400, max(1, q // 3)], dim, page, heads, group,
            window, sinks, holes=holes)


@pytest.mark.parametrize("dim,page,heads,group,q", ROWS)
def test_bounds_of_lengths(dim, page, heads, group, q):
    """Keys past max_kv and queries past max_q are left out."""
    for max_kv in (40, 1100):
        run([11, dim, q, max_kv], [q, 1, q], [1500, 60, 1101], dim, page, heads, group, max_kv=max_kv)
        run([12, dim, q, max_kv], [q, 1, q], [1500, 60, 1101], dim, page, heads, group, 50, 6, max_kv=max_kv)
    run([13, dim, q], [q + 9, 1, q], [1300, 60, 700], dim, page, heads, group, max_q=q)


# ---- large scales ------------------------------------------------------------------
@pytest.mark.parametrize("dim,page,heads,group,q", ROWS)
@pytest.mark.parametrize("scale,sharp", [(1e9, 2.0 ** -14), (-2e10, 2.0 ** -18), (1e-20, 1.0)])
def test_scales_of_any_size(dim, page, heads, group, q, scale, sharp):
    """A scale that is large and queries that are small: rows whose first steps,
    or all keys, are masked stay what they are."""
    run([14, dim, q], [q, q + 5, 1], [1500, max(1, q // 2), 40], dim, page, heads, group, scale=scale, sharp=sharp)
    run([15, dim, q], [q, q], [1500, 300 + q], dim, page, heads, group, 20, 2, scale=scale, sharp=sharp)


# ---- many tokens -------------------------------------------------------------------
def test_store_more_tokens_than_workgroups():
    """More than 2^24 tokens in one call leave what two calls leave."""
    T, dim, page = 2 ** 24 + 1000, 64, 256
    n = -(-T // page)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((T, dim), generator=g, device="cuda", dtype=torch.float16)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    slots = torch.arange(T, device="cuda")
    inv = dev((10000.0 ** (-np.arange(dim // 2) / (dim // 2))).astype(np.float32))
    gain = torch.linspace(0.5, 1.5, dim, device="cuda")
    outs = []
    for parts in ((0, T), (0, T // 2, T)):
        pages = torch.zeros((n, B.pn_kv4_page_bytes(page, 1, dim)), dtype=torch.uint8, device="cuda")
        q = torch.zeros_like(x)
        cache = B.KV4Cache(pages, n, page, 1, dim)
        for lo, hi in zip(parts, parts[1:]):
            say("store tokens %d..%d" % (lo, hi))
            B.pn_kv4_store(cache, hi - lo, x[lo:], x[lo:], x[lo:], "f16", dim, dim, dim, 1, gain, gain, 1e-6, inv, dim,
                           False, pos[lo:], slots[lo:], q[lo:], dim)
        sync()
        outs.append((pages, q))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert outs[0][1][-1].abs().max() > 0 and outs[0][0][(T - 1) // page].any()
