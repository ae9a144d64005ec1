"""Cases that measure the attention side of the decode path: the operators
that sit between the packed products of a decoder layer (q, k, v in, o out)
and after its head, each in a plain form (elementary torch operations) and as
the library's entry points.

Four operators:
  plan    pn_kv4_plan     slots, positions and block table of a ragged batch
  store   pn_kv4_store    norm of each query and key head, position rotation,
                          keys and values into the 4-bit cache (read back with
                          pn_kv4_load, so that the result holds values)
  attn    pn_kv4_attn     attention over the paged 4-bit cache: single tokens,
                          drafts to verify, prompt chunks, sliding windows
                          with first tokens that stay visible
  verify  pn_spec_verify  drafted tokens against the target's probabilities

The cache holds pn4t blocks (64 four-bit codes, one signed fp16 scale, value
d * (n - 8)).  A page holds `page` tokens; for each key-value head it has
  K codes   page rows of D/8 words; a row keeps its words in the order
            [g][b][h] of natural word 8 b + 4 h + g (b: block, h < 2, g < 4)
  V codes   [token / 4][word][token % 4], words in natural order
  K scales  [token][block] fp16
  V scales  [token][block] fp16
Word w holds elements 8 w .. 8 w + 7; element j of a word sits in half (j & 1)
at bit 4 (j >> 1) of that half.

The head shapes are the three ways to cut the 6144 query and 1024 key and
value columns of the sweep's layer into heads of 64, 128 or 256.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 64
Q_COLS, KV_COLS = 6144, 1024


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one verification step of a small batch: eight tokens for each of 16 requests
        dict(name="plan-drafts", op="plan", batch=16, page=16, ctx=8192, new=8, prompts=0),
        # a full server: thousands of decoding requests, one in sixteen brings a prompt
        dict(name="plan-server", op="plan", batch=4000, page=64, ctx=20000, new=8, prompts=2048),
        # the one token of one request, straight from the fp32 products
        dict(name="store-token", op="store", tokens=1, dim=256, page=64, half=False, rot=64, pairs=False, far=60000),
        # drafts of a batch, fp16 inputs, neighbouring pairs rotated
        dict(name="store-drafts", op="store", tokens=509, dim=64, page=16, half=True, rot=64, pairs=True, far=8000),
        # a long prompt
        dict(name="store-prompt", op="store", tokens=8191, dim=128, page=64, half=False, rot=128, pairs=False, far=131072),
        # one request deep in a long context: everything hangs on the split over the keys
        dict(name="attn-token", op="attn", batch=1, q=1, kv=65536, dim=256, page=64, ragged=False, window=0, sinks=0),
        # ordinary decoding of a ragged batch
        dict(name="attn-tokens", op="attn", batch=64, q=1, kv=16384, dim=128, page=16, ragged=True, window=0, sinks=0),
        # verification of seven drafts and the token before them
        dict(name="attn-drafts", op="attn", batch=16, q=8, kv=5003, dim=256, page=32, ragged=True, window=0, sinks=0),
        # a prompt of its own
        dict(name="attn-prompt", op="attn", batch=1, q=4096, kv=4096, dim=128, page=64, ragged=False, window=0, sinks=0),
        # later chunks of three long prompts under a window, the first tokens kept
        dict(name="attn-window", op="attn", batch=3, q=1000, kv=20000, dim=64, page=64, ragged=True, window=2048, sinks=4),
        # one request, seven drafts, a sharded head's vocabulary
        dict(name="verify-one", op="verify", batch=1, drafts=7, vocab=62080, probs=True),
        # a batch against the whole vocabulary, draft probabilities known
        dict(name="verify-batch", op="verify", batch=64, drafts=7, vocab=248320, probs=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "store", "attn", "attn", "verify"))
    if op == "plan":
        return dict(op=op, batch=_log(rng, 1, 4000), page=rng.choice((16, 32, 64, 128, 256)), ctx=_log(rng, 1, 20000),
                    new=rng.randint(1, 16), prompts=rng.choice((0, _log(rng, 1, 2048))))
    if op == "store":
        dim = rng.choice((64, 128, 256))
        return dict(op=op, tokens=_log(rng, 1, 8191), dim=dim, page=rng.choice((16, 32, 64, 128, 256)),
                    half=rng.random() < 0.5, rot=rng.choice((dim, dim // 2, dim // 4)), pairs=rng.random() < 0.5,
                    far=_log(rng, 100, 1000000))
    if op == "attn":
        dim, page = rng.choice((64, 128, 256)), rng.choice((16, 32, 64, 128, 256))
        window, sinks = rng.choice(((0, 0), (0, 0), (_log(rng, 16, 4096), rng.randint(0, 16))))
        kind = rng.choice(("token", "drafts", "prompt"))
        if kind == "token":
            batch = _log(rng, 1, 64)
            return dict(op=op, batch=batch, q=1, kv=_log(rng, 1, min(65536, 1000000 // batch)), dim=dim, page=page,
                        ragged=rng.random() < 0.7, window=window, sinks=sinks)
        if kind == "drafts":
            batch, q = _log(rng, 1, 32), rng.randint(2, 16)
            return dict(op=op, batch=batch, q=q, kv=_log(rng, q, min(20000, 200000 // batch)), dim=dim, page=page,
                        ragged=rng.random() < 0.7, window=window, sinks=sinks)
        q = _log(rng, 17, 2000)
        return dict(op=op, batch=rng.randint(1, 3), q=q, kv=q + rng.choice((0, _log(rng, 1, 2000))), dim=dim, page=page,
                    ragged=rng.random() < 0.5, window=window, sinks=sinks)
    batch = _log(rng, 1, 64)
    return dict(op=op, batch=batch, drafts=rng.choice((1, 3, 7)), vocab=_log(rng, 1000, 248320),
                probs=rng.random() < 0.7)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lengths(g, n, lo, hi):
    """n lengths in lo..hi, spread over their logarithm."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return torch.exp(math.log(lo) + u * (math.log(hi + 1) - math.log(lo))).floor().clamp(lo, hi).to(torch.int32)


def _page_bytes(page, heads, dim):
    return page * heads * (dim + dim // 16)


def _half(x):
    """fp64 -> fp16, rounded once: by way of fp32 rounded to odd (a plain cast rounds twice)."""
    f = x.float()
    back = f.double()
    bits = f.view(torch.int32) - (back.abs() > x.abs()).int()
    return torch.where(back == x, f, (bits | 1).view(torch.float32)).to(torch.float16)


def _scale_and_codes(y):
    """pn4t blocks of the last axis: fp16 scales [..., D/64] and codes 0..15 [..., D]."""
    b = y.unflatten(-1, (-1, BLOCK))
    at = b.abs().argmax(-1, keepdim=True)
    top = b.gather(-1, at)
    d = _half((top.double() / -8).clamp(-65504, 65504))
    step = torch.where(d == 0, torch.ones_like(d), d).to(y.dtype)
    n = torch.where(d == 0, torch.zeros_like(b), torch.round(b / step)).clamp(-8, 7) + 8
    return d.squeeze(-1), n.flatten(-2).to(torch.int32)


def _words(n):
    """Codes [..., D] -> int32 words [..., D/8]."""
    n = n.unflatten(-1, (-1, 8))
    w = torch.zeros_like(n[..., 0])
    for j in range(8):
        w |= n[..., j] << (16 * (j & 1) + 4 * (j >> 1))
    return w


def _word_order(dim, device):
    """Natural word held at each place of a stored key row."""
    at = torch.arange(dim // 8, device=device)
    g, b, h = at // (dim // 32), at % (dim // 32) // 2, at % 2
    return 8 * b + 4 * h + g


def _fill_pages(g, pages, page, heads, dim):
    """A cache of normed keys and of values with a few strong channels."""
    cache = torch.empty(pages, _page_bytes(page, heads, dim), dtype=torch.uint8, device="cuda")
    gain = torch.exp(0.5 * torch.randn(heads, 1, dim, generator=g, device="cuda"))
    step = max(1, (1 << 26) // (page * heads * dim))
    order = _word_order(dim, "cuda")
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn(n, heads, page, dim, generator=g, device="cuda")
        ks, kc = _scale_and_codes(x * 1.2)
        kw = _words(kc)[..., order]
        x = torch.randn(n, heads, page, dim, generator=g, device="cuda")
        vs, vc = _scale_and_codes(x * gain * 0.5)
        vw = _words(vc).unflatten(2, (page // 4, 4)).transpose(-1, -2)
        parts = [t.contiguous().view(torch.uint8).reshape(n, heads, -1) for t in (kw, vw, ks, vs)]
        cache[p:p + n] = torch.cat(parts, -1).reshape(n, -1)
    return cache


def _budget(case):
    """Tokens that one step of a plan case has room for."""
    prompts = (case["batch"] // 16 + 1) * case["prompts"] / math.log(case["prompts"] + 1) if case["prompts"] else 0
    return (case["batch"] * case["new"] + int(prompts) + 63) // 64 * 64


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    dev = "cuda"
    if case["op"] == "plan":
        n, page = case["batch"], case["page"]
        s["ctx"] = _lengths(g, n, 1, case["ctx"])
        s["new"] = torch.full((n,), case["new"], dtype=torch.int32, device=dev)
        if case["prompts"]:
            first = torch.rand(n, generator=g, device=dev) < 1 / 16
            first[0] = True
            s["new"] = torch.where(first, _lengths(g, n, 1, case["prompts"]), s["new"])
            s["ctx"] = torch.where(first, torch.zeros_like(s["ctx"]), s["ctx"])
        # a step of a fixed size: requests past its budget of tokens wait, or bring a part of their prompt
        s["tokens"] = _budget(case)
        before = s["new"].cumsum(0) - s["new"]
        s["new"] = torch.minimum(s["new"], (s["tokens"] - before).clamp_min(0)).int()
        # rejected drafts leave some requests a page ahead of their tokens
        ahead = (torch.rand(n, generator=g, device=dev) < 0.1).to(torch.int32)
        s["held"] = (s["ctx"] + page - 1) // page + ahead
        s["max_pages"] = (case["ctx"] + max(case["new"], case["prompts"]) + page - 1) // page + 1
        taken = int(s["held"].sum())
        pool = torch.randperm(taken + s["tokens"] // page + n, generator=g, device=dev).to(torch.int32)
        s["free"] = pool[taken:].contiguous()
        table = torch.full((n, s["max_pages"]), -1, dtype=torch.int32, device=dev)
        mine = torch.arange(s["max_pages"], device=dev) < s["held"][:, None]
        table[mine] = pool[:taken]
        s["table"] = table
        for name, count in (("held_out", n), ("q_start", n + 1), ("kv_len", n), ("positions", s["tokens"]), ("info", 2)):
            s[name] = torch.zeros(count, dtype=torch.int32, device=dev)
        s["slots"] = torch.zeros(s["tokens"], dtype=torch.int64, device=dev)
    elif case["op"] == "store":
        n, dim, page = case["tokens"], case["dim"], case["page"]
        s["heads"], s["kv_heads"] = Q_COLS // dim, KV_COLS // dim
        kind = torch.float16 if case["half"] else torch.float32
        # one product writes all three side by side
        x = torch.randn(n, Q_COLS + 2 * KV_COLS, generator=g, device=dev) * 1.7
        x *= torch.exp(0.4 * torch.randn(Q_COLS + 2 * KV_COLS, generator=g, device=dev))
        s["x"] = x.to(kind)
        s["q_gain"] = 1 + 0.2 * torch.randn(dim, generator=g, device=dev)
        s["k_gain"] = 1 + 0.2 * torch.randn(dim, generator=g, device=dev)
        half = case["rot"] // 2
        s["inv_freq"] = (1e6 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)).float()
        first = int(torch.randint(0, case["far"], (1,), generator=g, device=dev))
        s["positions"] = torch.arange(first, first + n, device=dev, dtype=torch.int32)
        pages = (n + page - 1) // page + 3
        s["pages"] = pages
        s["cache"] = torch.zeros(pages, _page_bytes(page, s["kv_heads"], dim), dtype=torch.uint8, device=dev)
        perm = torch.randperm(pages, generator=g, device=dev)
        at = torch.arange(n, device=dev) + 2  # the request's earlier tokens take the first two places
        s["slots"] = perm[at // page] * page + at % page
        s["q_out"] = torch.zeros(n, Q_COLS, dtype=torch.float16, device=dev)
        s["k_out"] = torch.zeros(n, KV_COLS, device=dev)
        s["v_out"] = torch.zeros(n, KV_COLS, device=dev)
    elif case["op"] == "attn":
        n, dim, page = case["batch"], case["dim"], case["page"]
        heads = KV_COLS // dim
        s["heads"], s["kv_heads"], s["scale"] = Q_COLS // dim, heads, dim ** -0.5
        q_len = torch.full((n,), case["q"], dtype=torch.int32, device=dev)
        kv = torch.full((n,), case["kv"], dtype=torch.int32, device=dev)
        if case["ragged"] and n > 1:
            kv[1:] = _lengths(g, n - 1, max(1, case["q"]), case["kv"])
        s["kv_len"] = kv
        s["q_start"] = torch.cat((torch.zeros_like(q_len[:1]), q_len.cumsum(0).to(torch.int32)))
        s["total"] = n * case["q"]
        s["max_pages"] = (case["kv"] + page - 1) // page
        used = (kv + page - 1) // page
        pages = int(used.sum()) + 1
        s["cache"] = _fill_pages(g, pages, page, heads, dim)
        s["pages"] = pages
        s["table"] = torch.full((n, s["max_pages"]), -1, dtype=torch.int32, device=dev)
        mine = torch.arange(s["max_pages"], device=dev) < used[:, None]
        s["table"][mine] = torch.randperm(pages, generator=g, device=dev)[:pages - 1].to(torch.int32)
        s["query"] = (1.5 * torch.randn(s["total"], Q_COLS, generator=g, device=dev)).half()
        s["out"] = torch.zeros(s["total"], Q_COLS, dtype=torch.float16, device=dev)
        s["ws"] = torch.empty(64 << 20, dtype=torch.uint8, device=dev)  # one for all layers of a program
    else:
        n, k, vocab = case["batch"], case["drafts"], case["vocab"]
        s["target"] = torch.empty(n, k + 1, vocab, device=dev)
        s["draft"] = torch.empty(n, k, vocab, device=dev) if case["probs"] else None
        s["tokens"] = torch.zeros(n, k, dtype=torch.int32, device=dev)
        for b in range(n):
            logits = 2.5 * torch.randn(k + 1, vocab, generator=g, device=dev)
            s["target"][b] = torch.softmax(logits, -1)
            guess = torch.softmax(logits[:k] + 0.3 * torch.randn(k, vocab, generator=g, device=dev), -1)
            if case["probs"]:
                s["draft"][b] = guess
            u = torch.rand(k, vocab, generator=g, device=dev).clamp_min(1e-30)
            picked = (guess.log() - (-u.log()).log()) if case["probs"] else guess
            s["tokens"][b] = picked.argmax(-1).to(torch.int32)
        s["count"] = torch.randint(0, k + 1, (n,), generator=g, device=dev).clamp_min(min(k, 1)).to(torch.int32)
        s["count"][0] = k
        s["uniform"] = torch.rand(n, k + 1, generator=g, device=dev)
        s["out"] = torch.zeros(n, k + 1, dtype=torch.int32, device=dev)
        s["accepted"] = torch.zeros(n, dtype=torch.int32, device=dev)
        s["ws"] = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------
# the library's entry points
# ---------------------------------------------------------------------------
def _cache(s):
    from bit_quantized_decode_pn3t_amd import _binding as B
    return B.KV4Cache(s["cache"], s["pages"], s["page"], s["kv_heads"], s["dim"])


def _run_own(s):
    from bit_quantized_decode_pn3t_amd import _binding as B
    if s["op"] == "plan":
        B.pn_kv4_plan(s["ctx"], s["new"], s["held"], s["batch"], s["free"], s["free"].numel(), s["page"], s["table"],
                      s["max_pages"], s["max_pages"], s["held_out"], s["q_start"], s["kv_len"], s["positions"],
                      s["slots"], s["tokens"], s["info"])
        return {k: s[k] for k in ("table", "held_out", "q_start", "kv_len", "positions", "slots", "info")}
    if s["op"] == "store":
        cache, x = _cache(s), s["x"]
        width = x.shape[1]
        B.pn_kv4_store(cache, s["tokens"], x, x[:, Q_COLS:], x[:, Q_COLS + KV_COLS:], "f16" if s["half"] else "f32",
                       width, width, width, s["heads"], s["q_gain"], s["k_gain"], 1e-6, s["inv_freq"], s["rot"],
                       s["pairs"], s["positions"], s["slots"], s["q_out"], Q_COLS)
        B.pn_kv4_load(cache, s["slots"], s["tokens"], s["k_out"], s["v_out"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    if s["op"] == "attn":
        B.pn_kv4_attn(_cache(s), s["query"], Q_COLS, s["heads"], s["q_start"], s["kv_len"], s["table"], s["max_pages"],
                      s["batch"], s["total"], s["q"], s["kv"], s["scale"], s["window"], s["sinks"], s["out"], Q_COLS,
                      s["ws"], s["ws"].numel())
        return s["out"]
    draft = s["draft"]
    B.pn_spec_verify(s["target"], s["vocab"], draft, s["vocab"], s["tokens"], s["drafts"], s["count"], s["uniform"],
                     s["drafts"] + 1, s["batch"], s["drafts"], s["vocab"], s["out"], s["drafts"] + 1, s["accepted"],
                     s["ws"], s["ws"].numel())
    return {"out": s["out"], "accepted": s["accepted"]}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_plan(s):
    n, page, dev = s["batch"], s["page"], s["ctx"].device
    ctx, new = s["ctx"].long().clamp_min(0), s["new"].long().clamp_min(0)
    ends = new.cumsum(0)
    total = ends[-1:]
    start = torch.cat((torch.zeros_like(total), ends))
    need = (ctx + new + page - 1) // page
    take = (need - s["held"]).clamp_min(0)
    first = take.cumsum(0) - take
    free = s["free"].numel()
    col = torch.arange(s["max_pages"], device=dev)
    nth = first[:, None] + col - s["held"][:, None]
    fresh = (col >= s["held"][:, None]) & (col < need[:, None])
    got = torch.where(nth < free, s["free"][nth.clamp(0, free - 1)], -1)
    table = torch.where(fresh, got, s["table"])
    t = torch.arange(s["tokens"], device=dev)
    b = torch.searchsorted(ends, t, right=True).clamp_max(n - 1)
    real = t < total
    pos = ctx[b] + t - start[b]
    which = (pos // page).clamp(0, s["max_pages"] - 1)
    at = table[b, which].long()
    good = real & (at >= 0) & (pos // page < s["max_pages"])
    slots = torch.where(good, at * page + pos % page, -1)
    info = torch.stack((take.sum().clamp_max(free), total[0] - good.sum()))
    return {"table": table, "held_out": torch.maximum(need, s["held"].long()).int(), "q_start": start.int(),
            "kv_len": (ctx + new).int(), "positions": torch.where(real, pos, -1).int(), "slots": slots, "info": info.int()}


def _plain_turn(y, cos, sin, rot, pairs):
    """Rotate the first `rot` elements of each head by the position's angles."""
    cos, sin = cos[:, None], sin[:, None]
    head, rest = y[..., :rot], y[..., rot:]
    if pairs:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, rest), -1)


def _plain_norm(x, gain):
    return x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * gain


def _plain_values(y):
    d, n = _scale_and_codes(y)
    return (d.float()[..., None] * (n - 8).float().unflatten(-1, (-1, BLOCK))).flatten(-2)


def _plain_store(s):
    n, dim = s["tokens"], s["dim"]
    q, k, v = s["x"].split((Q_COLS, KV_COLS, KV_COLS), 1)
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos(), angle.sin()
    q = _plain_norm(q.float().view(n, -1, dim), s["q_gain"])
    q = _plain_turn(q, cos.float(), sin.float(), s["rot"], s["pairs"]).half().flatten(1)
    # keys and values in 64 bits: next to a border between two codes 32 bits pick either
    k = _plain_norm(k.double().reshape(n, -1, dim), s["k_gain"].double())
    k = _plain_turn(k, cos, sin, s["rot"], s["pairs"])
    return {"q": q, "k": _plain_values(k).flatten(1), "v": _plain_values(v.double().reshape(n, -1, dim)).flatten(1)}


def _plain_unpack(words):
    """int32 words [..., W] -> codes minus 8, fp32 [..., 8 W]."""
    shift = torch.tensor([16 * (j & 1) + 4 * (j >> 1) for j in range(8)], dtype=torch.int32, device=words.device)
    return (((words[..., None] >> shift) & 15) - 8).float().flatten(-2)


def _plain_attn(s):
    n, dim, page, heads = s["batch"], s["dim"], s["page"], s["kv_heads"]
    group, dev = s["heads"] // heads, s["cache"].device
    pages = s["table"].shape[1]
    raw = s["cache"][s["table"].long().clamp_min(0)].view(n, pages, heads, -1)
    half, few = page * dim // 2, page * dim // 32
    kw, vw, ks, vs = (t.contiguous() for t in raw.split((half, half, few, few), -1))
    back = torch.argsort(_word_order(dim, dev))
    kw = kw.view(torch.int32).view(n, pages, heads, page, dim // 8)[..., back]
    vw = vw.view(torch.int32).view(n, pages, heads, page // 4, dim // 8, 4).transpose(-1, -2).flatten(3, 4)

    def values(words, scales):
        d = scales.view(torch.float16).view(n, pages, heads, page, dim // BLOCK).float()
        x = _plain_unpack(words).unflatten(-1, (-1, BLOCK)) * d[..., None]
        return x.flatten(-2).transpose(1, 2).reshape(n, heads, pages * page, dim)

    q_len = s["q_start"].diff()
    row = torch.arange(s["q"], device=dev)
    at = (s["q_start"][:-1, None] + row).clamp_max(s["total"] - 1).long()
    q = s["query"].float()[at].view(n, s["q"], heads, group, dim).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = torch.matmul(q, values(kw, ks).transpose(-1, -2).contiguous()) * s["scale"]
    pos = (s["kv_len"] - q_len)[:, None] + row
    key = torch.arange(pages * page, device=dev)
    seen = (key <= pos[..., None]) & (s["table"] >= 0).repeat_interleave(page, 1)[:, None]
    if s["window"]:
        seen &= (key > pos[..., None] - s["window"]) | (key < s["sinks"])
    score = score.view(n, heads, group, s["q"], -1)
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(top.masked_fill_(top == -math.inf, 0.0)).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score.flatten(2, 3), values(vw, vs)).view(n, heads, group, s["q"], dim)
    out = torch.where(total > 0, out / total, torch.zeros_like(out)).permute(0, 3, 1, 2, 4).reshape(-1, Q_COLS)
    t = torch.arange(s["total"], device=dev)
    b = torch.searchsorted(s["q_start"][1:], t, right=True).clamp_max(n - 1)
    return out[b * s["q"] + t - s["q_start"][b]].half()


def _plain_verify(s):
    n, k, vocab, dev = s["batch"], s["drafts"], s["vocab"], s["target"].device
    tok = s["tokens"].long()
    p = s["target"][:, :k].gather(-1, tok[..., None]).squeeze(-1).double()
    q = s["draft"].gather(-1, tok[..., None]).squeeze(-1).double() if s["probs"] else torch.ones_like(p)
    live = torch.arange(k, device=dev) < s["count"][:, None]
    took = ((s["uniform"][:, :k].double() * q < p) & live).long().cumprod(1).sum(1)
    b = torch.arange(n, device=dev)
    row = s["target"][b, took]
    more = took < s["count"]
    at = took.clamp_max(k - 1)
    if s["probs"]:
        rest = row - s["draft"][b, at]
    else:
        rest = torch.where(torch.arange(vocab, device=dev) == tok[b, at][:, None], torch.zeros_like(row), row)
    rest = torch.where(more[:, None], rest, row)
    rest = torch.where((rest > 0) & rest.isfinite(), rest, torch.zeros_like(rest))
    row = torch.where((row > 0) & row.isfinite(), row, torch.zeros_like(row))
    rest = torch.where((rest > 0).any(1, keepdim=True), rest, row)
    total = rest.double().cumsum(1)
    over = total > s["uniform"][:, k:].double() * total[:, -1:]
    last = vocab - 1 - (rest > 0).flip(1).int().argmax(1)
    token = torch.where(over.any(1), over.int().argmax(1), torch.where((rest > 0).any(1), last, -1))
    col = torch.arange(k + 1, device=dev)
    out = torch.cat((tok, torch.full_like(tok[:, :1], -1)), 1)
    out = torch.where(col < took[:, None], out, torch.where(col == took[:, None], token[:, None], -1))
    return {"out": out.int(), "accepted": took.int()}


def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plain_plan, "store": _plain_store, "attn": _plain_attn, "verify": _plain_verify}[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _visible(case):
    """Query-key pairs, keys read and queries of a case, with ragged lengths at their mean."""
    n, q, kv, w = case["batch"], case["q"], case["kv"], case["window"]
    lo = max(1, q)
    mean = (kv - lo) / math.log(kv / lo) if case["ragged"] and n > 1 and kv > lo else kv
    pairs = keys = 0.0
    for length, count in ((kv, 1), (mean, n - 1)):
        first = length - q
        if w and w < length:
            keys += count * min(length, q + w + case["sinks"])
            pairs += count * sum(min(first + i + 1, w + min(case["sinks"], max(0, first + i + 1 - w))) for i in range(q))
        else:
            keys += count * length
            pairs += count * (q * first + q * (q + 1) / 2)
    return pairs, keys


def work(case):
    if case["op"] == "plan":
        n, page = case["batch"], case["page"]
        new = _budget(case)
        fresh = new / page
        return {"bytes": n * 4 * 3 + fresh * 8 + n * 4 * 3 + new * 12, "flops": 0}
    if case["op"] == "store":
        n = case["tokens"]
        wide = 2 if case["half"] else 4
        stored = 2 * KV_COLS * (1 + 1 / 16) / 2
        # the values come back in 32 bits beside what is stored
        return {"bytes": n * ((Q_COLS + 2 * KV_COLS) * wide + Q_COLS * 2 + stored + 2 * KV_COLS * 4 + 12),
                "flops": n * (Q_COLS + KV_COLS) * 8}
    if case["op"] == "attn":
        pairs, keys = _visible(case)
        row = 2 * KV_COLS * (1 + 1 / 16) / 2
        return {"bytes": keys * row + 2 * case["batch"] * case["q"] * Q_COLS * 2, "flops": 4.0 * pairs * Q_COLS}
    rows = 2 if case["probs"] else 1
    return {"bytes": case["batch"] * (case["vocab"] * 4 * rows + case["drafts"] * 16), "flops": 0}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_plan(s):
    page, width = s["page"], s["max_pages"]
    ctx, new, held = (s[k].cpu().tolist() for k in ("ctx", "new", "held"))
    free, table = s["free"].cpu().tolist(), s["table"].cpu().tolist()
    used, start, kv, pos, slots, keep, lost = 0, [0], [], [], [], [], 0
    for b in range(s["batch"]):
        need = -(-(ctx[b] + new[b]) // page)
        for c in range(held[b], need):
            entry = free[used] if used < len(free) else -1
            used += 1
            if c < width:
                table[b][c] = entry
        for t in range(new[b]):
            c, o = divmod(ctx[b] + t, page)
            entry = table[b][c] if c < width else -1
            lost += entry < 0
            if len(pos) < s["tokens"]:
                pos.append(ctx[b] + t)
                slots.append(entry * page + o if entry >= 0 else -1)
        start.append(start[-1] + new[b])
        kv.append(ctx[b] + new[b])
        keep.append(max(need, held[b]))
    pad = [-1] * (s["tokens"] - len(pos))
    whole = {"table": table, "held_out": keep, "q_start": start, "kv_len": kv, "positions": pos + pad,
             "info": [min(used, len(free)), lost]}
    got = {k: torch.tensor(v, dtype=torch.int32) for k, v in whole.items()}
    got["slots"] = torch.tensor(slots + pad, dtype=torch.int64)
    return got


def _exact_store(s):
    n, dim, rot = s["tokens"], s["dim"], s["rot"]
    x = s["x"].double()
    angle = torch.outer(s["positions"].double(), s["inv_freq"].double())
    turn = torch.polar(torch.ones_like(angle), angle)
    done = {}
    for name, lo, cols, gain in (("q", 0, Q_COLS, s["q_gain"]), ("k", Q_COLS, KV_COLS, s["k_gain"]),
                                 ("v", Q_COLS + KV_COLS, KV_COLS, None)):
        heads = []
        for h in range(cols // dim):
            y = x[:, lo + h * dim:lo + (h + 1) * dim]
            if gain is not None:
                y = y / torch.sqrt((y * y).sum(1, keepdim=True) / dim + 1e-6) * gain.double()
                if s["pairs"]:
                    z = torch.complex(y[:, 0:rot:2].contiguous(), y[:, 1:rot:2].contiguous()) * turn
                    y = torch.cat((torch.view_as_real(z).reshape(n, rot), y[:, rot:]), 1)
                else:
                    z = torch.complex(y[:, :rot // 2].contiguous(), y[:, rot // 2:rot].contiguous()) * turn
                    y = torch.cat((z.real, z.imag, y[:, rot:]), 1)
            if name != "q":
                parts = []
                for b in range(0, dim, BLOCK):
                    blk = y[:, b:b + BLOCK]
                    hi, lo_ = blk.max(1).values, blk.min(1).values
                    big = torch.maximum(hi, -lo_)
                    # the sign is that of the first element that reaches the largest magnitude
                    first = (blk.abs() == big[:, None]).int().argmax(1)
                    d = (blk[torch.arange(n, device=blk.device), first] / -8).cpu().numpy().astype(np.float16)
                    d = torch.from_numpy(d).to(blk.device).double()[:, None]
                    parts.append(torch.where(d == 0, torch.zeros_like(blk), (blk / d).round().clamp(-8, 7) * d))
                y = torch.cat(parts, 1)
            heads.append(y)
        done[name] = torch.cat(heads, 1)
    return done


def _exact_attn(s):
    dim, page, heads = s["dim"], s["page"], s["kv_heads"]
    group = s["heads"] // heads
    out = torch.zeros(s["total"], Q_COLS, dtype=torch.float64, device="cuda")
    starts, lens = s["q_start"].cpu().tolist(), s["kv_len"].cpu().tolist()
    per = page * (dim + dim // 16)
    # byte and nibble of element e of a row: word e // 8, half j & 1, nibble j >> 1
    e = torch.arange(dim, device="cuda")
    j, w = e % 8, e // 8
    byte, low = 2 * (j & 1) + (j >> 2), ((j >> 1) & 1) * 4
    place = (w % 4) * (dim // 32) + (w // 8) * 2 + (w % 8) // 4
    t = torch.arange(page, device="cuda")[:, None]
    k_at = t * (dim // 2) + place * 4 + byte
    v_at = page * dim // 2 + ((t // 4) * (dim // 8) + w) * 16 + (t % 4) * 4 + byte
    for b in range(s["batch"]):
        length, q0, q1 = lens[b], starts[b], starts[b + 1]
        count = -(-length // page)
        bytes_ = s["cache"].view(s["pages"], heads, per)[s["table"][b, :count].long()]
        pos = torch.arange(length - (q1 - q0), length, device="cuda")
        key = torch.arange(length, device="cuda")
        for h in range(heads):
            raw = bytes_[:, h]
            sc = raw[:, page * dim:].contiguous().view(torch.float16).double().view(count, 2, page, dim // BLOCK)

            def get(at, which):
                n = (raw[:, at] >> low.to(torch.uint8)) & 15
                d = sc[:, which].repeat_interleave(BLOCK, -1)
                return ((n.double() - 8) * d).view(-1, dim)[:length]

            k, v = get(k_at, 0), get(v_at, 1)
            for g in range(group):
                col = (h * group + g) * dim
                score = s["query"][q0:q1, col:col + dim].double() @ k.T * s["scale"]
                hide = key > pos[:, None]
                if s["window"]:
                    hide |= (key <= pos[:, None] - s["window"]) & (key >= s["sinks"])
                score[hide] = -math.inf
                out[q0:q1, col:col + dim] = torch.softmax(score, -1) @ v
    return out


def _exact_verify(s):
    n, k, vocab = s["batch"], s["drafts"], s["vocab"]
    outs, counts = torch.full((n, k + 1), -1, dtype=torch.int32), torch.zeros(n, dtype=torch.int32)
    toks, many, uni = s["tokens"].cpu().tolist(), s["count"].cpu().tolist(), s["uniform"].double().cpu().tolist()
    for b in range(n):
        i = 0
        while i < many[b]:
            p = float(s["target"][b, i, toks[b][i]])
            q = float(s["draft"][b, i, toks[b][i]]) if s["probs"] else 1.0
            if not uni[b][i] * q < p:
                break
            outs[b, i] = toks[b][i]
            i += 1
        w = s["target"][b, i].clone()
        if i < many[b]:
            if s["probs"]:
                w -= s["draft"][b, i]
            else:
                w[toks[b][i]] = 0
        w = w.double().clamp_min(0)
        if float(w.sum()) == 0:
            w = s["target"][b, i].double()
        c = torch.cumsum(w, 0)
        place = int(torch.searchsorted(c, c[-1:] * uni[b][k], right=True)[0])
        outs[b, i] = place if place < vocab else int(w.nonzero()[-1])
        counts[b] = i
    return {"out": outs, "accepted": counts}


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "store": _exact_store, "attn": _exact_attn, "verify": _exact_verify}[case["op"]](s)
