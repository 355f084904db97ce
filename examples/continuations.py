"""Many continuations of one prompt, by one attention layer with random weights.

The prompt goes into the paged 8-bit cache once.  Every continuation's page table begins with the prompt's full pages;
the tokens of its last, partly filled page are read back and appended to a page of each continuation's own.  A
step then appends a token to every continuation, attends with the common pages read once, and draws the next
tokens from the logits.  A step is captured in a CUDA graph and replayed.

    python examples/continuations.py --prompt 32768 --samples 128 --steps 32 --top-p 0.95
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from indexer_topk_long_gb300 import PagedKVCache, sample  # noqa: E402


def rotation_tables(positions: int, dim: int, base: float = 10000.0):
    angles = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, dim, 2) / dim)
    return angles.cos().float().cuda(), angles.sin().float().cuda()


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


class Continuations:
    """The layer, its cache, and the state of all continuations."""

    def __init__(self, prompt: int, samples: int, steps: int, q_heads: int, kv_heads: int, dim: int, page: int, vocabulary: int,
                 hidden: int, seed: int, settings: dict):
        rng = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=rng, device="cuda", dtype=torch.float32)
        self.q_heads, self.kv_heads, self.dim, self.settings = q_heads, kv_heads, dim, settings
        width = (q_heads + 2 * kv_heads) * dim
        self.embedding = normal(vocabulary, hidden).bfloat16()
        self.w_qkv = (normal(hidden, width) * hidden ** -0.5).bfloat16()
        self.w_out = (normal(q_heads * dim, hidden) * (q_heads * dim) ** -0.5).bfloat16()
        self.w_head = (normal(hidden, vocabulary) * hidden ** -0.5).bfloat16()
        self.u = torch.rand((steps + 1, samples), generator=rng, device="cuda")
        full, tail = divmod(prompt, page)
        own = -(-(tail + steps) // page)
        self.cache = PagedKVCache(full + 1 + samples * own, kv_heads, dim, page=page)
        pages = torch.randperm(full + 1 + samples * own, generator=rng, device="cuda").to(torch.int32)
        self.prompt_table = pages[None, :full + 1].contiguous()
        self.table = torch.cat([pages[:full].expand(samples, -1), pages[full + 1:].view(samples, own)], 1).contiguous()
        self.cos, self.sin = rotation_tables(prompt + steps, dim)
        self.cu = torch.arange(samples + 1, dtype=torch.int32, device="cuda")
        # the prompt, once
        x = self.embedding[torch.randint(0, vocabulary, (prompt,), generator=rng, device="cuda")]
        q, k, v = self.project(x)
        held, whole = ints([prompt]), ints([0, prompt])
        q = self.cache.append(k, v, self.prompt_table, held, whole, self.cos, self.sin, q=q)
        out, _ = self.cache.attention(q[-1:], self.prompt_table, held, ints([0, 1]), max_q=1)
        # its last page's tokens to a page of each continuation's own, as they are held
        if tail:
            k, v = self.cache.read(self.prompt_table, held, ints([0, tail]), tail)
            self.cache.append(k.repeat(samples, 1, 1), v.repeat(samples, 1, 1), self.table, ints([prompt] * samples), self.cu * tail)
        # what every step changes: the first tokens come from the prompt's last logits
        self.lens = ints([prompt] * samples)
        self.at = torch.zeros(1, dtype=torch.long, device="cuda")
        self.token, self.logp = sample(self.logits(x[-1:], out).expand(samples, -1).contiguous(), self.u[0], **settings)

    def project(self, x):
        y = (x @ self.w_qkv).view(len(x), -1, self.dim)
        return y.split([self.q_heads, self.kv_heads, self.kv_heads], 1)

    def logits(self, x, out):
        return ((x + out.flatten(1) @ self.w_out) @ self.w_head).float()

    def step(self):
        """One token for every continuation."""
        x = self.embedding[self.token.long()]
        q, k, v = self.project(x)
        self.lens += 1
        self.at += 1
        q = self.cache.append(k, v, self.table, self.lens, self.cu, self.cos, self.sin, q=q)
        out, _ = self.cache.attention_shared(q, self.table, self.lens, self.cu, max_q=1)
        sample(self.logits(x, out), self.u[self.at][0], **self.settings, token=self.token, logp=self.logp)


def run(prompt: int, samples: int, steps: int, q_heads: int = 32, kv_heads: int = 8, dim: int = 128, page: int = 64,
        vocabulary: int = 32768, hidden: int = 1024, seed: int = 0, graph: bool = True, **settings):
    """Returns the continuations' tokens [samples, steps + 1], the logarithms of their probabilities, and milliseconds a step."""
    state = Continuations(prompt, samples, steps, q_heads, kv_heads, dim, page, vocabulary, hidden, seed, settings)
    tokens, logps = [state.token.clone()], [state.logp.clone()]
    advance = state.step
    if graph and steps > 1:
        state.step()                     # the first by itself, to warm up
        tokens.append(state.token.clone())
        logps.append(state.logp.clone())
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            state.step()
        advance = captured.replay
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    n = steps + 1 - len(tokens)
    for _ in range(n):
        advance()
        tokens.append(state.token.clone())
        logps.append(state.logp.clone())
    t1.record()
    torch.cuda.synchronize()
    if state.cache.status() != 0:
        raise RuntimeError("the cache reports an error")
    return torch.stack(tokens, 1), torch.stack(logps, 1), t0.elapsed_time(t1) / max(n, 1), state


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("prompt", 32768), ("samples", 128), ("steps", 32), ("q-heads", 32), ("kv-heads", 8), ("dim", 128), ("page", 64),
                        ("vocabulary", 131072), ("hidden", 1024), ("top-k", 0)):
        p.add_argument("--" + name, type=int, default=value)
    for name, value in (("temperature", 0.8), ("top-p", 0.95), ("min-p", 0.0)):
        p.add_argument("--" + name, type=float, default=value)
    tokens, logps, ms, _ = run(**vars(p.parse_args()))
    print("%d continuations of %d tokens: %.3f ms a step, mean log-probability %.3f, %d different ones" % (
        *tokens.shape, ms, float(logps.mean()), len(torch.unique(tokens, dim=0))))


if __name__ == "__main__":
    main()
