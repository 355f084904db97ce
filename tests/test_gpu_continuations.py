"""Append, read, shared attention and sampling together: the example that continues one prompt in many ways."""
import importlib.util
import os

import pytest

import sampling_reference as ref

pytestmark = pytest.mark.gpu
SIZES = dict(vocabulary=5000, hidden=64)


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "continuations.py")
    spec = importlib.util.spec_from_file_location("continuations", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("prompt,q_heads,kv_heads,dim,page", [(700, 8, 2, 128, 64), (333, 4, 4, 64, 16), (256, 14, 2, 64, 32)])
def test_a_graph_gives_the_bits_of_single_calls(prompt, q_heads, kv_heads, dim, page):
    import torch
    ex = _example()
    sizes = dict(prompt=prompt, samples=9, steps=20, q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=page, **SIZES)
    settings = dict(temperature=1.2, top_k=200, top_p=0.97)
    tokens, logps, _, state = ex.run(**sizes, **settings)
    again = ex.run(**sizes, **settings, graph=False)
    assert torch.equal(tokens, again[0]) and torch.equal(logps, again[1])
    assert tokens.shape == (9, 21) and bool((tokens >= 0).all()) and bool(logps.isfinite().all())
    assert len(torch.unique(tokens, dim=0)) == 9


@pytest.mark.parametrize("prompt", [640, 700, 13])
def test_forks_hold_the_prompt(prompt):
    """What a continuation holds of the prompt is what the prompt's own pages hold."""
    import torch
    ex = _example()
    samples = 5
    state = ex.run(prompt=prompt, samples=samples, steps=3, q_heads=4, kv_heads=2, dim=64, page=32, **SIZES)[3]
    want = state.cache.read(state.prompt_table, ex.ints([prompt]), ex.ints([0, prompt]), prompt)
    got = state.cache.read(state.table, ex.ints([prompt] * samples), state.cu * prompt, samples * prompt)
    for a, b in zip(want, got):
        assert torch.equal(a.repeat(samples, 1, 1), b)
    assert state.cache.status() == 0


def test_a_step_by_its_parts():
    """The attention of a step against that of every sequence by itself, and its tokens against the reference of
    the sampler on the step's logits."""
    import torch
    ex = _example()
    settings = dict(temperature=0.9, top_p=0.9)
    state = ex.run(prompt=1000, samples=12, steps=5, q_heads=8, kv_heads=2, dim=128, page=64, **SIZES, **settings, graph=False)[3]
    q = torch.randn((12, 8, 128), device="cuda").bfloat16()
    out, lse = state.cache.attention_shared(q, state.table, state.lens, state.cu, max_q=1)
    want, want_lse = state.cache.attention(q, state.table, state.lens, state.cu, max_q=1)
    # both within an output's rounding (2^-8) and f16 weights (2^-11, twice) of the exact one
    assert float((out.float() - want.float()).abs().max() / want.float().abs().max()) < 2 * (2.0 ** -8 + 2.0 ** -10)
    assert float((lse - want_lse).abs().max()) < 2.0 ** -9
    x = state.embedding[state.token.long()]
    logits, u = state.logits(x, out), state.u[3]
    ref.check(logits, u, ex.sample(logits, u, **settings), **settings)


def test_greedy_continuations_agree():
    """Without chance all continuations of a prompt are the same."""
    import torch
    ex = _example()
    tokens, logps, _, _ = ex.run(prompt=500, samples=7, steps=8, q_heads=8, kv_heads=2, dim=128, page=64, **SIZES, temperature=0.0)
    assert torch.equal(tokens, tokens[:1].expand_as(tokens)) and bool((logps == 0).all())
