"""Plain 64-bit implementations of the attention-side operators, numpy only
(test helper): the paged pn4t cache's layout, the batch plan, norm + rotation
+ store, attention, draft verification.  Written from include/pn.h's text."""
import numpy as np

from oracle import pnref

BLOCK = 64


def page_bytes(page, heads, dim):
    return page * heads * (dim + dim // 16)


def half(x):
    """fp64 -> fp16, saturated."""
    return np.clip(np.asarray(x, np.float64), -65504, 65504).astype(np.float16)


def quantize(y):
    """[..., dim] fp64 -> (scales fp16 [..., dim/64], codes [..., dim])."""
    y = np.asarray(y, np.float64)
    b = y.reshape(y.shape[:-1] + (-1, BLOCK))
    mag = np.where(np.isnan(b), -1.0, np.abs(b))
    top = np.take_along_axis(b, mag.argmax(-1)[..., None], -1)
    top = np.where(np.isnan(top), 0.0, top)
    d = half(-top / 8)
    d = np.where(d == 0, np.float16(0), d)
    step = np.where(d == 0, 1.0, d.astype(np.float64))
    with np.errstate(invalid="ignore"):
        n = np.clip(np.rint(b / step), -8, 7)
    n = np.where(np.isnan(b) | (d == 0), 0, n)
    return d[..., 0], (n + 8).astype(np.int64).reshape(y.shape)


def value(scales, codes):
    d = np.repeat(scales.astype(np.float64), BLOCK, -1)
    return d * (codes - 8)


def _places(dim):
    """Byte offset in a K row, and low bit, of each element; word and the rest for V."""
    e = np.arange(dim)
    w, j = e // 8, e % 8
    b, h, g = w // 8, (w % 8) // 4, w % 4
    place = g * (dim // 32) + 2 * b + h
    bit = 16 * (j & 1) + 4 * (j >> 1)
    return place, w, bit // 8, bit % 8


def put(pages, page, heads, dim, slot, side, scales, codes):
    """Write one token (scales [heads, dim/64], codes [heads, dim]) into uint8 pages [P, bytes]."""
    place, w, byte, low = _places(dim)
    p, o = divmod(int(slot), page)
    R = dim // BLOCK
    for h in range(heads):
        base = h * page * (dim + dim // 16)
        if side == "k":
            at = base + o * dim // 2 + 4 * place + byte
            sc = base + page * dim + 2 * o * R
        else:
            at = base + page * dim // 2 + 4 * (((o // 4) * (dim // 8) + w) * 4 + o % 4) + byte
            sc = base + page * dim + 2 * page * R + 2 * o * R
        for a, n, s in zip(at, codes[h], low):
            pages[p, a] = (int(pages[p, a]) & (0xF0 if s == 0 else 0x0F)) | (int(n) << s)
        pages[p, sc:sc + 2 * R] = np.ascontiguousarray(scales[h].astype(np.float16)).view(np.uint8)


def get(pages, page, heads, dim, slots):
    """Values of slots: k, v [T, heads, dim] fp64 (and their fp16 scales and codes)."""
    place, w, byte, low = _places(dim)
    slots = np.asarray(slots, np.int64)
    p, o = slots // page, slots % page
    R = dim // BLOCK
    out = []
    for side in "kv":
        val = np.zeros((len(slots), heads, dim))
        for h in range(heads):
            base = h * page * (dim + dim // 16)
            if side == "k":
                at = base + o[:, None] * (dim // 2) + (4 * place + byte)[None]
                sc = base + page * dim + 2 * o * R
            else:
                at = base + page * dim // 2 + 4 * ((o[:, None] // 4 * (dim // 8) + w) * 4 + o[:, None] % 4) + byte
                sc = base + page * dim + 2 * page * R + 2 * o * R
            n = (pages[p[:, None], at].astype(np.int64) >> low) & 15
            d = pages[p[:, None], sc[:, None] + np.arange(2 * R)]
            with np.errstate(invalid="ignore"):  # unwritten scales may be NaN
                val[:, h] = value(np.ascontiguousarray(d).view(np.float16), n)
        out.append(val)
    return out


def store(x, heads_of, gains, eps, inv_freq, rot, pairs, positions, dim):
    """Normed and rotated q, k (fp64) of x = (q, k) rows."""
    done = []
    pos = np.asarray(positions, np.float64)
    angle = pos[:, None] * np.asarray(inv_freq, np.float64)[None] if rot else None
    for rows, heads, gain in zip(x, heads_of, gains):
        y = np.asarray(rows, np.float64).reshape(len(rows), heads, dim)
        if gain is not None:
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * np.asarray(gain, np.float64)
        y = y.copy()
        if rot:
            c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
            if pairs:
                a, b = y[..., 0:rot:2].copy(), y[..., 1:rot:2].copy()
                y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
            else:
                a, b = y[..., :rot // 2].copy(), y[..., rot // 2:rot].copy()
                y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, a * s + b * c
        done.append(y)
    return done


def attend(q, pages, page, heads, dim, q_start, kv_len, table, scale, window, sinks, num_pages):
    """q [T, q_heads, dim] -> (out, bound): fp64 outputs, and for each what an
    fp32 pass with one fp16 rounding of each weight, of each value and of the
    output may be off by."""
    T, q_heads, _ = q.shape
    group = q_heads // heads
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    q = q.astype(np.float64)
    for b in range(len(kv_len)):
        n, q0, q1 = max(0, int(kv_len[b])), int(q_start[b]), int(q_start[b + 1])
        if q1 <= q0 or n == 0:
            continue
        t = np.arange(n)
        entry = np.asarray(table[b])[np.minimum(t // page, table.shape[1] - 1)]
        there = (entry >= 0) & (entry < num_pages)
        k, v = get(pages, page, heads, dim, np.where(there, entry, 0).astype(np.int64) * page + t % page)
        for i in range(q0, q1):
            p = n - (q1 - q0) + i - q0
            see = there & (t <= p)
            if window > 0:
                see &= (t > p - window) | (t < sinks)
            if not see.any():
                continue
            for h in range(q_heads):
                kk, vv = k[see, h // group], v[see, h // group]
                s = kk @ q[i, h] * scale
                mag = (np.abs(kk) @ np.abs(q[i, h])) * abs(scale)
                w = np.exp(s - s.max())
                out[i, h] = w @ vv / w.sum()
                a = w @ np.abs(vv) / w.sum()
                # scores: dim products and a few scalings in fp32; exp2 of a difference of two scores
                eta = 2 * ((dim + 8) * 2.0 ** -24 * mag.max() + 8 * 2.0 ** -24)
                e = a * (2 * 2.0 ** -11 + 2 * eta + (see.sum() + 64) * 2.0 ** -24)
                e += see.sum() * np.abs(vv).max() * 2.0 ** -34  # weights below fp16's normal range
                bound[i, h] = e + 2.0 ** -11 * (np.abs(out[i, h]) + e) + 2.0 ** -25
    return out, bound


def plan(ctx, new, held, free, page, table, max_pages, max_tokens):
    table = np.array(table)
    used, start, kv, keep, pos, slots, lost = 0, [0], [], [], [], [], 0
    for b in range(len(ctx)):
        c, n, h = (max(0, int(x[b])) for x in (ctx, new, held))
        need = -(-(c + n) // page)
        for col in range(h, need):
            if col < max_pages:
                table[b, col] = free[used] if used < len(free) else -1
            used += 1
        for t in range(n):
            col, o = divmod(c + t, page)
            entry = int(table[b, col]) if col < max_pages else -1
            if len(pos) < max_tokens:
                pos.append(c + t)
                slots.append(entry * page + o if entry >= 0 else -1)
                lost += entry < 0
            else:
                lost += 1
        start.append(start[-1] + n)
        kv.append(c + n)
        keep.append(max(h, need))
    pad = [-1] * (max_tokens - len(pos))
    return dict(table=table, held_out=keep, q_start=start, kv_len=kv, positions=pos + pad, slots=slots + pad,
                info=[min(used, len(free)), lost])


def verify(target, draft, tokens, n_draft, u):
    """target [B, k+1, V], draft [B, k, V] or None; fp32 arrays."""
    B, k1, V = target.shape
    out, acc = np.full((B, k1), -1, np.int32), np.zeros(B, np.int32)

    def clean(x):
        with np.errstate(invalid="ignore"):
            return np.where((x > 0) & np.isfinite(x), x, 0).astype(np.float64)

    for b in range(B):
        n = k1 - 1 if n_draft is None else min(max(int(n_draft[b]), 0), k1 - 1)
        a = 0
        while a < n:
            x = int(tokens[b, a])
            if not 0 <= x < V:
                break
            p = float(target[b, a, x])
            q = 1.0 if draft is None else float(draft[b, a, x])
            if not float(u[b, a]) * q < p:
                break
            out[b, a] = x
            a += 1
        row = target[b, a]
        if a < n:
            if draft is not None:
                with np.errstate(invalid="ignore"):
                    r = clean(row - draft[b, a])
            else:
                r = clean(row)
                if 0 <= tokens[b, a] < V:
                    r[tokens[b, a]] = 0
        else:
            r = clean(row)
        if not (r > 0).any():
            r = clean(row)
        if (r > 0).any():
            c = np.cumsum(r)
            over = np.nonzero(c > float(u[b, k1 - 1]) * c[-1])[0]
            out[b, a] = over[0] if len(over) else np.nonzero(r > 0)[0][-1]
        acc[b] = a
    return out, acc


def pnref_codes(y):
    """The C oracle's pn4t quantizer on fp32 rows [N, dim]: (scales, codes)."""
    n, dim = y.shape
    raw = pnref.quantize("pn4t", np.ascontiguousarray(y, np.float32), n, dim).reshape(n, dim // BLOCK, 34)
    d = np.ascontiguousarray(raw[..., :2]).view(np.float16)[..., 0]
    words = np.ascontiguousarray(raw[..., 2:]).view(np.uint32)
    j = np.arange(8)
    n_ = (words[..., None] >> (16 * (j & 1) + 4 * (j >> 1)).astype(np.uint32)) & 15
    return d, n_.reshape(n, dim).astype(np.int64)
