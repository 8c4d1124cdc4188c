"""Best of n over a small linear-attention model: a prompt is read once, its state branched n ways, every branch
sampled token by token and scored by its own log probabilities, and all but the best give their pages back.

    python examples/best_of_n.py [--branches 8] [--steps 16]

The model is a random one of generic shape (embedding, two layers of linear attention with a decay per head,
a language-model head); what it shows is how the serving calls go together:

    linattn_prefill   the prompt, into the page of slot 0
    pages_fork        branches share that page: nothing is copied
    pages_own         each branch gets a page of its own ...
    linattn_decode    ... and its first token goes from the shared page into it, later ones on from there
    token_logprobs    the sampled tokens' log probabilities and the distribution's entropy
    pages_free, pages_compact   the losers' pages, and the winner's moved to the front
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import exact_replay_decode_gb300 as ers  # noqa: E402


class Model:
    """tokens -> logits, with one LinAttnCache per layer."""

    def __init__(self, vocab=5003, width=1024, layers=2, heads=8, groups=4, dim=128, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, device="cuda", generator=g) * shape[0] ** -0.5).to(torch.bfloat16)

        self.heads, self.groups, self.dim = heads, groups, dim
        self.embed = torch.randn(vocab, width, device="cuda", generator=g).to(torch.bfloat16)
        self.layers = [(weight(width, 2 * groups * dim + heads * dim), weight(heads * dim, width)) for _ in range(layers)]
        self.head = weight(width, vocab)
        self.decay = -torch.exp2(-8.0 * torch.arange(1, heads + 1, dtype=torch.float32, device="cuda") / heads)

    def caches(self, slots, pages):
        return [ers.LinAttnCache(slots, self.heads, self.groups, self.dim, self.dim, npages=pages) for _ in self.layers]

    def __call__(self, tokens, attend):
        """attend(layer, q, k, v) -> o, the cache's part."""
        x = self.embed[tokens]
        for n, (w_in, w_out) in enumerate(self.layers):
            y = torch.nn.functional.rms_norm(x, x.shape[-1:]) @ w_in
            q, k, v = y.split([self.groups * self.dim] * 2 + [self.heads * self.dim], dim=1)
            q, k = (torch.nn.functional.normalize(t.view(-1, self.groups, self.dim).float(), dim=-1).to(x.dtype)
                    for t in (q, k))
            o = attend(n, q.contiguous(), k.contiguous(), v.reshape(-1, self.heads, self.dim).contiguous())
            x = x + o.reshape(len(x), -1) @ w_out
        return torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.head


def best_of_n(model, prompt, branches=8, steps=16, temperature=0.8, seed=0):
    """(tokens of the best branch, scores of all, the caches, the branches' tokens)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    caches = model.caches(1 + branches, 1 + branches)
    root = torch.zeros(1, dtype=torch.int32, device="cuda")
    kids = torch.arange(1, 1 + branches, dtype=torch.int32, device="cuda")
    for c in caches:
        ers.pages_own(c.pages, root)
    logits = model(prompt, lambda n, q, k, v: ers.linattn_prefill(caches[n], q, k, v, model.decay, slot=root))[-1:]
    read = []
    for c in caches:
        ers.pages_fork(c.pages, root.repeat(branches), kids)
        read.append(ers.pages_own(c.pages, kids, copy=False))
    logits = logits.expand(branches, -1)
    score = torch.zeros(branches, device="cuda")
    tokens = []
    for step in range(steps):
        p = torch.softmax(logits.float() / temperature, -1)
        token = torch.multinomial(p, 1, generator=gen)[:, 0]
        logprob, entropy, top_id, top_logprob = ers.token_logprobs(logits.contiguous(), token.to(torch.int32), top_k=4)
        score += logprob
        tokens.append(token)
        logits = model(token, lambda n, q, k, v: ers.linattn_decode(caches[n], q, k, v, model.decay, kids,
                                                                    read_page=read[n] if step == 0 else None))
    best = int(score.argmax())
    losers = kids[torch.arange(branches, device="cuda") != best].contiguous()
    for c in caches:
        ers.pages_free(c.pages, losers)
        ers.pages_compact(c.pages)
    tokens = torch.stack(tokens, 1)
    return tokens[best], score, caches, tokens


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--branches", type=int, default=8)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    model = Model()
    prompt = torch.randint(0, len(model.embed), (300,), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    tokens, score, caches, _ = best_of_n(model, prompt, a.branches, a.steps)
    print("scores  ", " ".join(f"{s:.2f}" for s in score.tolist()))
    print("best    ", tokens.tolist())
    print("pages in use", [int((c.pages.refs > 0).sum()) for c in caches], "of", caches[0].npages)


if __name__ == "__main__":
    main()
