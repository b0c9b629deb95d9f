"""Speculative decoding with the drafter around a small target model of random weights: every call
of the step in the order in which an engine makes them.

    propose -> update_state -> target over the last token and the draft (KVCache.write,
    KVCache.attend in every layer) -> verify -> accept_feedback -> propose ...

The verifier's outputs are the drafter's inputs, so the loop reads nothing back to the host.

    python examples/verify_step.py [--steps N] [--greedy]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import suffix_match_drafter_amd as sfx  # noqa: E402


class Target:
    """Pre-norm attention blocks over an 8-bit paged cache; every second layer looks at a window
    and a few first tokens only."""

    def __init__(self, vocab, layers=2, heads=8, kv_heads=2, dim=64, window=128, sinks=4, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g, device="cuda") * shape[0] ** -0.5).bfloat16()

        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.width = heads * dim
        self.embed = weight(vocab, self.width) * vocab ** 0.5
        self.layers = [dict(qkv=weight(self.width, (heads + 2 * kv_heads) * dim),
                            out=weight(self.width, self.width),
                            up=weight(self.width, 2 * self.width),
                            down=weight(2 * self.width, self.width),
                            window=window if i % 2 else 0, sinks=sinks if i % 2 else 0)
                       for i in range(layers)]
        self.head = weight(self.width, vocab)

    def caches(self, pages, page):
        return [sfx.KVCache(pages, page, self.kv_heads, self.dim) for _ in self.layers]

    def __call__(self, ids, caches, table, start, count):
        """Logits [B, T, V] of tokens ids [B, T] at positions start[b] + 0, 1, ..., of which
        count[b] are real."""
        B, T = ids.shape
        q_cols, kv_cols = self.heads * self.dim, self.kv_heads * self.dim
        x = self.embed[ids.clamp(min=0).long()]
        for layer, cache in zip(self.layers, caches):
            qkv = torch.nn.functional.rms_norm(x, (self.width,)) @ layer["qkv"]
            q, k, v = qkv.split((q_cols, kv_cols, kv_cols), 2)     # strided views, used as they are
            cache.write(k.unflatten(2, (self.kv_heads, self.dim)),
                        v.unflatten(2, (self.kv_heads, self.dim)), table, start, count)
            o = cache.attend(q.unflatten(2, (self.heads, self.dim)), table, start + count, count,
                             window=layer["window"], sinks=layer["sinks"])
            x = x + o.flatten(2) @ layer["out"]
            h = torch.nn.functional.rms_norm(x, (self.width,))
            x = x + torch.nn.functional.silu(h @ layer["up"]) @ layer["down"]
        return torch.nn.functional.rms_norm(x, (self.width,)) @ self.head


def decode(steps=40, greedy=False, batch=8, vocab=1000, prompt=96, k=8, page=64, seed=0):
    """Decodes `steps` steps; returns the tokens [B, S], their lengths [B] and the accepted counts
    [steps, B], all on the device."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    most = prompt + 1 + steps * (k + 1)
    width = -(-(most + k) // page)
    target = Target(vocab, seed=seed)
    caches = target.caches(batch * width, page)
    table = torch.randperm(batch * width, generator=g, device="cuda").int().view(batch, width)
    drafter = sfx.Drafter(sfx.Config(k=k, max_tree_depth=8, max_batch=batch, max_seq=most,
                                     max_sampled=k + 1))
    # prompts that repeat themselves, so that there is something to match
    tokens = torch.zeros((batch, most), dtype=torch.int32, device="cuda")
    tokens[:, :prompt] = torch.randint(0, vocab, (batch, 24), generator=g, device="cuda",
                                       dtype=torch.int32).repeat(1, prompt // 24 + 1)[:, :prompt]
    temperature = torch.full((batch,), 0.0 if greedy else 0.7, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    # the prompt in one go, and the first token: a verification of an empty draft
    lens = torch.full((batch,), prompt, dtype=torch.int32, device="cuda")
    logits = target(tokens[:, :prompt], caches, table, torch.zeros_like(lens), lens)
    empty = torch.empty((batch, 0), dtype=torch.int32, device="cuda")
    first, _ = sfx.verify(logits[:, -1:], empty, None, uniform(batch, 0), uniform(batch),
                          temperature)
    sampled = torch.full((batch, k + 1), -1, dtype=torch.int32, device="cuda")
    sampled[:, :1] = first

    accepted = []
    for _ in range(steps):
        draft, num_valid = drafter.propose(lens, tokens, sampled)
        lens = sfx.update_state(tokens, lens, sampled)
        last = tokens.gather(1, (lens - 1).long()[:, None])
        logits = target(torch.cat([last, draft], 1), caches, table, lens - 1, num_valid + 1)
        sampled, num_accepted = sfx.verify(logits, draft, num_valid, uniform(batch, k),
                                           uniform(batch), temperature)
        drafter.accept_feedback(num_accepted)
        accepted.append(num_accepted)
    lens = sfx.update_state(tokens, lens, sampled)
    drafter.close()
    return tokens, lens, torch.stack(accepted)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=40)
    p.add_argument("--greedy", action="store_true")
    a = p.parse_args()
    tokens, lens, accepted = decode(a.steps, a.greedy)
    torch.cuda.synchronize()
    print(f"{a.steps} steps of {tokens.shape[0]} requests: lengths {lens.tolist()}, "
          f"{accepted.float().mean().item():.2f} drafted tokens accepted a step and request")


if __name__ == "__main__":
    main()
