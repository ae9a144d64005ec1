"""Speculative decoding steps over packed weights and the packed cache: the
attention-side operators as a decoder uses them, next to the products.

A small random decoder (attention layers and a head, all matrices pn4t; the
embedding, the norm of the hidden state, residual sums and softmax are plain
torch) answers a ragged batch of requests.  One step takes each request's last
token and k drafted ones:
  pn_kv4_plan      slots, positions and block table of the step's tokens
  per layer        q, k, v products; pn_kv4_store; pn_kv4_attn; o product
  pn_spec_verify   accepts drafts against the head's probabilities and draws
                   the next token
and the requests' lengths grow by what was accepted.  Prompts are the same
step with their own lengths, and k = 0 is token-by-token decoding.  Lengths
stay on the device; nothing in a step waits for the GPU.

A prompt that all requests begin with is entered once (Requests.share); from
then on pn_kv4_attn_shared reads its pages once for all of them.  With
sandwich=True a layer's output is normed and gated before it enters the
stream, and pn_residual_norm does all that lies between two layers' products.
Requests.score gives the answers' log probabilities, the entropy and the most
probable alternatives (pn_logprobs).

  python -m bit_quantized_decode_pn3t_amd.spec_step [--layers 4] [--batch 8] [--drafts 7] ...
"""
import argparse
import time

import numpy as np
import torch

from . import _binding as B
from . import synth

SMALL_M = 16  # pn_gemm_smallm's largest M; more rows take pn_gemm_prefill


def norm(h):
    return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6)


def product(W, n, k, x):
    """fp32 [M, n] of fp16 x [M, k] and a packed pn4t matrix."""
    m = x.shape[0]
    y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    run = B.pn_gemm_smallm if m <= SMALL_M else B.pn_gemm_prefill
    run("pn4t", W, n, k, x, x.stride(0), m, y, n)
    return y


class Decoder:
    """Random weights of one shape.  mix: what a layer's output is multiplied
    by; the less, the more of the drafts (which see the embedding alone) pass.
    sandwich: a layer's output y enters the stream as mix * sigmoid(z) *
    norm(y), with z a product of the layer's input."""

    def __init__(self, layers, hidden, q_heads, heads, dim, vocab, window=0, sinks=0, mix=1.0, seed=0, device="cuda",
                 sandwich=False):
        self.mix, self.sandwich = mix, sandwich
        self.hidden, self.q_heads, self.heads, self.dim, self.vocab = hidden, q_heads, heads, dim, vocab
        self.window, self.sinks, self.device = window, sinks, torch.device(device)
        g = np.random.default_rng(seed)

        def packed(n, k):
            return torch.from_numpy(synth.random_blocks(g, "pn4t", n, k)).to(self.device)

        q, kv = q_heads * dim, heads * dim
        self.layers = [dict(q=packed(q, hidden), k=packed(kv, hidden), v=packed(kv, hidden), o=packed(hidden, q))
                       for _ in range(layers)]
        if sandwich:
            for w in self.layers:
                w["gate"] = packed(hidden, hidden)
                w["post"] = torch.from_numpy(1 + 0.2 * g.standard_normal(hidden).astype(np.float32)).to(self.device)
        self.head = packed(vocab, hidden)
        self.embed = torch.from_numpy(g.standard_normal((vocab, hidden)).astype(np.float32)).to(self.device)
        self.gain = torch.ones(dim, device=self.device)
        self.rot = dim
        self.inv_freq = (10000.0 ** (-torch.arange(0, dim, 2, device=self.device).double() / dim)).float()

    def logits(self, h):
        """Of hidden states, or (fp16) of their norms."""
        return product(self.head, self.vocab, self.hidden, h if h.dtype == torch.float16 else norm(h).half())

    def draft(self, last, k, noise):
        """k drafts a request by the head on the embedding alone, with their
        probabilities [B, k, vocab]; noise: exponential, [k, B, vocab]."""
        rows, tokens = [], []
        for j in range(k):
            p = torch.softmax(self.logits(self.embed[last.long()]), -1)
            last = (p / noise[j]).argmax(-1).int()
            rows.append(p)
            tokens.append(last)
        return torch.stack(tokens, 1), torch.stack(rows, 1)


class Requests:
    """A batch of requests of at most max_len tokens: their caches (one a
    layer, sharing one block table), lengths and last tokens."""

    def __init__(self, model, batch, max_len, page_size=64):
        self.model, self.batch, self.page_size = model, batch, page_size
        self.max_pages = -(-max_len // page_size)
        self.max_len = self.max_pages * page_size
        dev = self.device = model.device
        n = batch * self.max_pages
        size = n * B.pn_kv4_page_bytes(page_size, model.heads, model.dim)
        self.caches = [B.KV4Cache(torch.empty(size, dtype=torch.uint8, device=dev), n, page_size, model.heads,
                                  model.dim) for _ in model.layers]
        # page ids, -1 behind them: a request that is given none loses its tokens, and no page goes to two
        self.free = torch.cat((torch.arange(n, dtype=torch.int32), torch.tensor([-1], dtype=torch.int32))).to(dev)
        self.order = torch.arange(n + 1, device=dev)
        self.lost = torch.zeros((), dtype=torch.int32, device=dev)  # tokens that found no place
        self.longest = 0  # at least every request's tokens, known without waiting for the GPU
        i32 = dict(dtype=torch.int32, device=dev)
        self.table = torch.full((batch, self.max_pages), -1, **i32)
        self.ctx, self.held, self.last = (torch.zeros(batch, **i32) for _ in range(3))
        self.kv_len, self.q_start = torch.empty(batch, **i32), torch.empty(batch + 1, **i32)
        self.info = torch.empty(2, **i32)
        self.ws = torch.empty(0, dtype=torch.uint8, device=dev)
        self.prefix = None  # pages [1, n] that all requests begin with

    def _room(self, max_q):
        """Refuse a step that could bring a request past max_len.  Its table
        row ends there: tokens past it would not reach the cache, and pages
        taken for them would be lost.  Near the end the lengths themselves are
        read, which waits for the GPU."""
        if self.longest + max_q > self.max_len:
            self.longest = int(self.ctx.max())
        if self.longest + max_q > self.max_len:
            raise ValueError("%d more tokens for a request of %d pass max_len = %d" % (max_q, self.longest, self.max_len))
        self.longest += max_q

    def check(self):
        """Raise if a token of any step so far found no place in the cache (waits for the GPU)."""
        if int(self.lost):
            raise RuntimeError("%d tokens found no place in the cache" % int(self.lost))

    def share(self, tokens):
        """Enter a prompt that all requests begin with, before any other
        tokens: its whole pages, once.  Returns how many tokens that were; the
        rest belongs in front of each request's own prompt."""
        n = tokens.numel() // self.page_size
        if self.longest or self.prefix is not None:
            raise ValueError("a shared prompt comes first")
        if n == 0:
            return 0
        if self.model.window:
            raise ValueError("a window does not see a shared prompt")
        count = n * self.page_size
        self._room(count)
        new = torch.zeros(self.batch, dtype=torch.int32, device=self.device)
        new[0] = count
        self._forward(tokens[:count], new, count)
        self.table[:, :n] = self.table[0, :n].clone()
        self.ctx, self.held = torch.full_like(self.ctx, count), torch.full_like(self.held, n)
        self.prefix = self.table[:1, :n].clone()
        self.shared = torch.tensor([n], dtype=torch.int32, device=self.device)
        self.g_start = torch.tensor([0, self.batch], dtype=torch.int32, device=self.device)
        return count

    def _attend(self, cache, q16, out, T, max_q):
        m, q_row = self.model, self.model.q_heads * self.model.dim
        args = (cache, q16, q_row, m.q_heads, self.q_start, self.kv_len, self.table, self.max_pages, self.batch)
        if self.prefix is None:
            B.pn_kv4_attn(*args, T, max_q, self.max_len, m.dim ** -0.5, m.window, m.sinks, out, q_row, self.ws,
                          self.ws.numel())
        else:
            n = self.prefix.shape[1]
            B.pn_kv4_attn_shared(*args, self.g_start, self.prefix, n, self.shared, 1, T, max_q, self.max_len, n,
                                 m.dim ** -0.5, out, q_row, self.ws, self.ws.numel())

    def _between(self, h, y, z, w, x):
        """y of layer w, gated by z, into the stream h, and the stream's norm into x."""
        m, n = self.model, self.model.hidden
        B.pn_residual_norm(h.shape[0], n, h, n, y, n, "f32", "sigmoid" if y is not None else "none", z, n, y is not None,
                           w["post"] if w else None, m.mix, None, None, 1e-6, h if y is not None else None, n, x, n)

    def _forward(self, tokens, new_len, max_q):
        """Hidden states [T, hidden] of the step's tokens, which enter the
        cache; of a sandwich decoder their norms, fp16."""
        m, dev, T = self.model, self.device, tokens.numel()
        positions = torch.empty(T, dtype=torch.int32, device=dev)
        slots = torch.empty(T, dtype=torch.int64, device=dev)
        held = torch.empty_like(self.held)
        B.pn_kv4_plan(self.ctx, new_len, self.held, self.batch, self.free, self.free.numel(), self.page_size,
                      self.table, self.max_pages, self.max_pages, held, self.q_start, self.kv_len, positions, slots, T,
                      self.info)
        self.held = held
        self.lost += self.info[1]
        self.free = self.free[(self.order + self.info[0]).clamp_(max=self.order.numel() - 1)]

        q_row, kv_row = m.q_heads * m.dim, m.heads * m.dim
        if self.prefix is None:
            need = B.pn_kv4_attn_workspace(self.caches[0], m.q_heads, self.batch, T, max_q, self.max_len, m.window,
                                           m.sinks)
        else:
            need = B.pn_kv4_attn_shared_workspace(self.caches[0], m.q_heads, self.batch, 1, T, max_q, self.max_len,
                                                  self.prefix.shape[1])
        if self.ws.numel() < need:
            self.ws = torch.empty(need, dtype=torch.uint8, device=dev)
        q16 = torch.empty((T, q_row), dtype=torch.float16, device=dev)
        out = torch.empty_like(q16)
        # a drafted token outside the vocabulary is refused later, and read as one inside
        h = m.embed[tokens.long().clamp(0, m.vocab - 1)]
        if m.sandwich:
            x = torch.empty((T, m.hidden), dtype=torch.float16, device=dev)
            self._between(h, None, None, None, x)
        for w, cache in zip(m.layers, self.caches):
            if not m.sandwich:
                x = norm(h).half()
            q, k, v = (product(w[name], n, m.hidden, x) for name, n in (("q", q_row), ("k", kv_row), ("v", kv_row)))
            B.pn_kv4_store(cache, T, q, k, v, "f32", q_row, kv_row, kv_row, m.q_heads, m.gain, m.gain, 1e-6,
                           m.inv_freq, m.rot, False, positions, slots, q16, q_row)
            self._attend(cache, q16, out, T, max_q)
            y = product(w["o"], m.hidden, q_row, out)
            if m.sandwich:
                self._between(h, y, product(w["gate"], m.hidden, m.hidden, x), w, x)
            else:
                h = h + m.mix * y
        return x if m.sandwich else h

    def _answer(self, h, tokens, draft, u, k, greedy):
        m = self.model
        logits = m.logits(h)
        if greedy:
            p = torch.zeros_like(logits).scatter_(1, logits.argmax(1, keepdim=True), 1.0)
        else:
            p = torch.softmax(logits, -1)
        out = torch.empty((self.batch, k + 1), dtype=torch.int32, device=self.device)
        accepted = torch.empty(self.batch, dtype=torch.int32, device=self.device)
        ws = torch.empty(B.pn_spec_workspace(self.batch, m.vocab), dtype=torch.uint8, device=self.device)
        B.pn_spec_verify(p, m.vocab, draft, m.vocab, tokens, max(k, 1), None, u, k + 1, self.batch, k, m.vocab, out,
                         k + 1, accepted, ws, ws.numel())
        self.last = out.gather(1, accepted[:, None].long())[:, 0]
        return out, accepted, logits

    def score(self, logits, tokens, top=0, scale=1.0):
        """ln p of tokens [rows, n] in softmax(scale * logits), the rows'
        entropies, and the `top` most probable tokens with their ln p.
        logits: fp32 or fp16 [rows, vocab]."""
        rows, n = tokens.shape
        dev, vocab = self.device, self.model.vocab
        kind = {torch.float32: "f32", torch.float16: "f16"}.get(logits.dtype)
        if kind is None or logits.shape != (rows, vocab):
            raise ValueError("scores of %d rows need fp32 or fp16 logits [%d, %d], not %s %s"
                             % (rows, rows, vocab, logits.dtype, list(logits.shape)))
        if logits.stride(1) != 1 or logits.stride(0) < vocab:
            logits = logits.contiguous()
        tokens = torch.where((tokens >= 0) & (tokens < vocab), tokens, -1).int().contiguous()
        logp, entropy = torch.empty((rows, n), device=dev), torch.empty(rows, device=dev)
        ids, best = torch.empty((rows, top), dtype=torch.int32, device=dev), torch.empty((rows, top), device=dev)
        ws = torch.empty(B.pn_logprobs_workspace(rows, vocab, top), dtype=torch.uint8, device=dev)
        B.pn_logprobs(logits, kind, logits.stride(0), rows, vocab, scale, tokens, n, n, logp, n, entropy, top,
                      ids if top else None, best if top else None, top, ws, ws.numel())
        return logp, entropy, ids, best

    def prompt(self, tokens, lengths, u, greedy=False):
        """Prompts (one flat row of tokens; lengths on the host, 1 and up) into
        the cache and each request's first token; u: [batch, 1]."""
        if len(lengths) != self.batch or min(lengths) < 1 or sum(lengths) != tokens.numel():
            raise ValueError("%d tokens for prompts of %s" % (tokens.numel(), lengths))
        self._room(max(lengths))
        new = torch.tensor(lengths, dtype=torch.int32, device=self.device)
        h = self._forward(tokens, new, max(lengths))
        self.ctx = self.kv_len.clone()
        none = torch.zeros((self.batch, 1), dtype=torch.int32, device=self.device)
        return self._answer(h[self.q_start[1:].long() - 1], none, None, u, 0, greedy)

    def step(self, u, tokens=None, draft=None, greedy=False):
        """Verify k drafted tokens [batch, k] (with their probabilities
        [batch, k, vocab], or None for a drafter that is certain) and draw one
        more each; u: [batch, k + 1].  Returns out, accepted and the logits."""
        k = 0 if tokens is None else tokens.shape[1]
        self._room(k + 1)
        row = self.last[:, None] if k == 0 else torch.cat((self.last[:, None], tokens), 1)
        new = torch.full((self.batch,), k + 1, dtype=torch.int32, device=self.device)
        h = self._forward(row.reshape(-1), new, k + 1)
        out, accepted, logits = self._answer(h, row if k == 0 else tokens, draft, u, k, greedy)
        self.ctx = self.ctx + accepted + 1  # rejected drafts are written over by the next step
        return out, accepted, logits


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("layers", 4), ("hidden", 5120), ("q-heads", 24), ("heads", 4), ("dim", 256),
                        ("vocab", 32768), ("window", 0), ("sinks", 0), ("batch", 8), ("prompt", 700), ("drafts", 7),
                        ("steps", 20), ("seed", 0), ("shared", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--mix", type=float, default=0.02)
    ap.add_argument("--sandwich", action="store_true")
    ap.add_argument("--score", action="store_true", help="the tokens' mean ln p and entropy")
    a = ap.parse_args()
    model = Decoder(a.layers, a.hidden, a.q_heads, a.heads, a.dim, a.vocab, a.window, a.sinks, a.mix,
                    a.seed, sandwich=a.sandwich)
    dev = model.device
    g = np.random.default_rng(a.seed)
    lengths = [int(n) for n in g.integers(1, a.prompt + 1, a.batch)]
    req = Requests(model, a.batch, a.shared + max(lengths) + (a.steps + 2) * (a.drafts + 1))
    rand = torch.Generator(device=dev)
    rand.manual_seed(a.seed)

    def uniform(k):
        return torch.rand((a.batch, k + 1), generator=rand, device=dev)

    if a.shared:
        common = torch.from_numpy(g.integers(0, a.vocab, a.shared, dtype=np.int32)).to(dev)
        a.shared = req.share(common)
    req.prompt(torch.from_numpy(g.integers(0, a.vocab, sum(lengths), dtype=np.int32)).to(dev), lengths, uniform(0))
    noise = torch.empty((max(a.drafts, 1), a.batch, a.vocab), device=dev)
    total = torch.zeros((), dtype=torch.int64, device=dev)
    sums = torch.zeros(2, dtype=torch.float64, device=dev)
    for i in range(a.steps + 1):
        if i == 1:  # the first step is for warming up
            torch.cuda.synchronize()
            total.zero_(), sums.zero_()
            t0 = time.perf_counter()
        tokens = draft = None
        if a.drafts:
            tokens, draft = model.draft(req.last, a.drafts, noise.exponential_(generator=rand))
        out, accepted, logits = req.step(uniform(a.drafts), tokens, draft)
        total += accepted.sum() + a.batch
        if a.score:
            logp, entropy, _, _ = req.score(logits, out.reshape(-1, 1))
            given = out.reshape(-1) >= 0
            sums += torch.stack([torch.where(given, x, 0.0).double().sum() for x in (logp[:, 0], entropy)])
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) / max(a.steps, 1) * 1e3
    req.check()
    print("%d requests, %sprompts of %d..%d tokens, %d layers: %.2f tokens a request and step (1 to %d), %.2f ms a step"
          % (a.batch, "%d shared tokens and " % a.shared if a.shared else "", min(lengths), max(lengths), a.layers,
             int(total) / max(a.steps, 1) / a.batch, a.drafts + 1, ms))
    if a.score:
        print("a token's ln p: %.3f, its distribution's entropy: %.3f" % tuple((sums / total).tolist()))


if __name__ == "__main__":
    main()
