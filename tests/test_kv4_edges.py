"""Refusals of the attention-side entry points and of the example at their
edges, on the CPU: every call here fails its host checks before any launch."""
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


def requests(monkeypatch, max_len, lengths):
    """The example's requests on the CPU, with steps that only count."""
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace
    from bit_quantized_decode_pn3t_amd import spec_step as S
    model = SimpleNamespace(device=torch.device("cpu"), heads=1, dim=64, layers=[0])
    req = S.Requests(model, len(lengths), max_len, 16)
    ran = []
    monkeypatch.setattr(S.Requests, "_forward", lambda self, tokens, new_len, max_q: ran.append(max_q) or torch.zeros(8, 4))
    monkeypatch.setattr(S.Requests, "_answer", lambda self, *a: (None, torch.zeros(len(lengths), dtype=torch.int32), None))
    req.kv_len, req.q_start = torch.tensor(lengths, dtype=torch.int32), torch.ones(len(lengths) + 1, dtype=torch.int32)
    return torch, req, ran


def test_example_refuses_steps_past_max_len(monkeypatch):
    """A request that would pass its table row is refused before anything runs."""
    torch, req, ran = requests(monkeypatch, 30, [20, 27])  # two pages: 32
    assert req.max_len == 32
    none = torch.zeros((2, 1), dtype=torch.int32)
    with pytest.raises(ValueError):
        req.prompt(torch.zeros(60, dtype=torch.int32), [33, 27], none)
    assert ran == []
    req.prompt(torch.zeros(47, dtype=torch.int32), [20, 27], none)
    for _ in range(3):  # drafts refused each time: one token a step, 27 -> 30, though 27 + 3 * 3 > 32
        req.step(none, torch.zeros((2, 2), dtype=torch.int32))
    assert req.ctx.tolist() == [23, 30] and ran == [27, 3, 3, 3]
    with pytest.raises(ValueError):
        req.step(none, torch.zeros((2, 2), dtype=torch.int32))
    req.step(none, torch.zeros((2, 1), dtype=torch.int32))
    req.step(none)
    with pytest.raises(ValueError):
        req.step(none)
    assert req.ctx.tolist() == [25, 32] and len(ran) == 6


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_attn_refuses_scales_that_are_not_finite(scale):
    cache = B.KV4Cache(BASE, 4, 16, 2, 64)
    args = dict(q=BASE, ldq=256, q_heads=4, q_start=BASE, kv_len=BASE, table=BASE, ld_table=8, B=3, total_q=0, max_q=2,
                max_kv=100, window=0, sinks=0, out=BASE, ldo=256, ws=None, ws_bytes=0, stream=0, check=False)
    assert B.pn_kv4_attn(cache, scale=scale, **args) == ESHAPE
    assert B.pn_kv4_attn(cache, scale=3.4e38, **args) == 0  # no queries: nothing to launch


def test_pages_past_2_gib_are_refused():
    """A page's bytes are 32-bit offsets in attention."""
    for heads, dim, page, status in ((65535, 256, 256, EUNSUPPORTED), (30841, 256, 256, EUNSUPPORTED), (30840, 256, 256, 0),
                                     (65535, 128, 256, EUNSUPPORTED), (65535, 64, 256, 0)):
        cache = B.KV4Cache(BASE, 2, page, heads, dim)
        assert B.pn_kv4_page_bytes(page, heads, dim) == page * heads * (dim + dim // 16)
        assert B.pn_kv4_load(cache, BASE, 0, BASE, BASE, stream=0, check=False) == status
        assert B.pn_kv4_attn(cache, BASE, heads * dim, heads, BASE, BASE, BASE, 8, 1, 0, 1, 100, 1.0, 0, 0, BASE,
                             heads * dim, None, 0, stream=0, check=False) == status


def test_load_refuses_more_than_a_launch_holds():
    cache = B.KV4Cache(BASE, 4, 16, 2, 64)  # 16 words a token
    for tokens in (2 ** 28, 2 ** 40):
        assert B.pn_kv4_load(cache, BASE, tokens, BASE, None, stream=0, check=False) == EUNSUPPORTED


@pytest.mark.parametrize("lengths,count", [([0, 9], 9), ([4, 5], 8), ([9], 9), ([3, 3, 3], 9), ([10, -1], 9)])
def test_example_refuses_prompts_that_do_not_fit(monkeypatch, lengths, count):
    """A prompt without tokens has no last token to answer from."""
    torch, req, ran = requests(monkeypatch, 30, [20, 27])
    with pytest.raises(ValueError):
        req.prompt(torch.zeros(count, dtype=torch.int32), lengths, torch.zeros((2, 1)))
    assert ran == []
