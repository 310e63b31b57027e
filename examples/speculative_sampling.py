"""A small hybrid language model with random weights that samples several continuations of each prompt, several tokens a step.

  python examples/speculative_sampling.py

Gated-delta layers (fp32 states in slots) and softmax attention layers (a quantized paged cache) take ragged prompts in chunks. Each prompt is
then forked into samples, which share its pages until they write. A draft model (a table of bigrams, of which the target's logits are a sum
with the layers') names a tree of tokens a step; the target runs over all of them at once, and its probabilities decide which path is kept.
Sampled tokens are distributed as the target's alone.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_gated_delta_gb300 as P  # noqa: E402

CHUNK, PAGE = 256, 64


def tree_bits(parents):
    """Depth of each node, and its ancestors (itself among them) as 32-bit words [N, ceil(N / 32)]; parents[i] < i, node 0 is the root."""
    N = len(parents)
    see, depth = torch.zeros(N, (N + 31) // 32 * 32, dtype=torch.int64), torch.zeros(N, dtype=torch.int32)
    for i in range(N):
        if i:
            see[i], depth[i] = see[parents[i]], depth[parents[i]] + 1
        see[i, i] = 1
    words = (see.view(N, -1, 32) << torch.arange(32)).sum(-1)
    return depth, torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()


class Server:
    """`rows` sequences at most; all layers share one page table, one vector of lengths and the rows' numbers as slots."""

    def __init__(self, kinds, rows, max_tokens, vocab=512, heads=8, kv_heads=2, d=128, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda o, i: (torch.randn(o, i, generator=g, device="cuda") * i ** -0.5).bfloat16()
        self.rows, self.heads, self.kv_heads, self.d, self.dm, self.vocab = rows, heads, kv_heads, d, heads * d, vocab
        self.embed, self.unembed = w(vocab, self.dm) * self.dm ** 0.5, w(vocab, self.dm)
        self.bigrams = torch.randn(vocab, vocab, generator=g, device="cuda") * 2
        self.rope = P.PaceRope(d, max_tokens + CHUNK)
        cols = (max_tokens + CHUNK) // PAGE
        self.pages = P.PacePages(rows * cols, PAGE, rows)
        self.table = torch.full((rows, cols), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.layers = []
        for kind in kinds:
            if kind == "attend":
                kv = P.PaceKV(P.make_kv_config(heads, kv_heads, d, rows * cols, rows, page_tokens=PAGE, max_new=CHUNK))
                self.layers.append((kind, kv, w((heads + 2 * kv_heads) * d, self.dm), w(self.dm, self.dm), None))
            else:
                delta = P.PaceDelta(P.make_delta_config(heads, d, rows, key_heads=kv_heads))
                self.layers.append((kind, delta, w((heads + 2 * kv_heads) * d, self.dm), w(self.dm, self.dm), w(2 * heads, self.dm)))

    def forward(self, tokens, n_new, mask=None, depth=None):
        """Logits [B, T, vocab]. Prompt tokens advance the states; those of a tree (mask) leave them, and what they need to follow an accepted
        path is kept in self.drafts."""
        x = self.embed[tokens.long()]
        B, T, _ = x.shape
        self.drafts = []
        for kind, layer, wqkv, wo, wab in self.layers:
            h = torch.nn.functional.normalize(x.float(), dim=-1).mul(self.dm ** 0.5).to(x.dtype)
            q, k, v = (h @ wqkv.t()).view(B, T, -1, self.d).split(
                [self.heads, self.kv_heads, self.kv_heads] if kind == "attend" else [self.kv_heads, self.kv_heads, self.heads], 2)
            o = torch.empty(B, T, self.heads, self.d, dtype=x.dtype, device=x.device)
            if kind == "attend":
                qr = torch.empty_like(o)
                at = None if depth is None else self.lens[:, None] + depth
                layer.append(q, k, v, self.lens, self.table, rope=self.rope, positions=at, n_new=n_new, q_out=qr)
                layer.attend(qr, o, self.lens, self.table, mask=mask, n_new=n_new)
            else:
                q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(x.dtype) for t in (q, k))
                a, beta = torch.sigmoid((h @ wab.t()).float()).view(B, T, 2, self.heads).unbind(2)
                a = 1 - 0.1 * a
                if mask is None:
                    layer.chunk(q, k, v, a, beta, o, lens=self.lens, n_new=n_new)
                else:
                    layer.draft(q, k, v, a, beta, o, lens=self.lens, n_new=n_new, mask=mask)
                    self.drafts.append((layer, k, v, a, beta))
            x = x + o.flatten(2) @ wo.t()
        return (x @ self.unembed.t()).float() + self.bigrams[tokens.long()]

    def take(self, n):
        """Pages for n[b] more tokens of each row; the last pages that rows still share are copied."""
        fits = torch.empty_like(n)
        self.pages.take(self.table, self.lens, n, fits)
        for kind, layer, *_ in self.layers:
            if kind == "attend":
                layer.copy_pages(self.pages)
        return fits

    def prompt(self, prompts):
        """Prompts (lists of tokens, empty for unused rows) but for their last tokens, which are returned."""
        n = torch.tensor([max(len(p) - 1, 0) for p in prompts], dtype=torch.int32, device="cuda")
        tokens = torch.zeros(self.rows, max(1, int(n.max())), dtype=torch.int32)
        for b, p in enumerate(prompts):
            tokens[b, :max(len(p) - 1, 0)] = torch.tensor(p[:-1], dtype=torch.int32)
        tokens = tokens.cuda()
        for t0 in range(0, tokens.shape[1], CHUNK):
            new = (n - t0).clamp(0, min(CHUNK, tokens.shape[1] - t0))
            self.take(new)
            self.forward(tokens[:, t0:t0 + CHUNK], new)
            self.lens += new
        return torch.tensor([p[-1] if p else 0 for p in prompts], dtype=torch.int32, device="cuda")

    def fork(self, src):
        """Row b goes on as a copy of row src[b] (-1: it is given up). Pages are shared; recurrent states are copied."""
        self.pages.select(self.table, self.lens, torch.tensor(src, dtype=torch.int32, device="cuda"))
        pick = torch.tensor(src, device="cuda").clamp(min=0)
        for kind, layer, *_ in self.layers:
            if kind != "attend":
                layer.states.copy_(layer.states[pick])

    def sample(self, token, live, steps, parents, g):
        """At least `steps` tokens of each live row, after `token` [rows]: lists, and the mean number of tokens a step."""
        N, dev = len(parents), token.device
        depth, bits = tree_bits(parents)
        depth, mask = depth.to(dev), bits.to(dev).expand(self.rows, -1, -1).contiguous()
        n_new = live.int() * N
        out, taken, used = [[] for _ in range(self.rows)], 0, 0
        while min(len(o) for o, on in zip(out, live.tolist()) if on) < steps:
            tree = torch.empty(self.rows, N, dtype=torch.int32, device=dev)
            tree[:, 0] = token
            q = torch.empty(self.rows, N, self.vocab, device=dev)
            for i in range(N):                               # drafts of one node are drawn independently of one another
                if i:
                    tree[:, i] = torch.multinomial(q[:, parents[i]], 1, generator=g)[:, 0]
                q[:, i] = torch.softmax(self.bigrams[tree[:, i].long()], -1)
            self.take(n_new)
            p = torch.softmax(self.forward(tree, n_new, mask, depth), -1)
            idx = torch.empty_like(tree)
            n_keep, following = torch.empty(2, self.rows, dtype=torch.int32, device=dev)
            P.pace_verify(tree, p, q, torch.rand(self.rows, N, generator=g, device=dev), idx, n_keep, following, mask=mask, n_new=n_new)
            for kind, layer, *_ in self.layers:
                if kind == "attend":
                    layer.keep(self.lens, self.table, idx, n_keep)
            for layer, *x in self.drafts:
                layer.keep(*x, idx, n_keep, lens=self.lens)  # (a row without tokens yet begins with a zero state)
            self.lens += n_keep
            self.pages.select(self.table, self.lens)         # pages of drafts that were not kept go back
            new = torch.cat((tree.gather(1, idx.long()), following[:, None]), 1).tolist()
            for b, n in enumerate(n_keep.tolist()):
                if n:
                    out[b] += new[b][1:n] + new[b][-1:]
                    taken, used = taken + n, used + 1
            token = torch.where(n_keep > 0, following, token)
        return out, taken / used

    def status(self):
        return [layer.status() for _, layer, *_ in self.layers] + [self.pages.status()]


def main(steps=24):
    rows, samples, vocab = 8, 4, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    server = Server(["delta", "attend", "delta"], rows, 1024)
    prompts = [torch.randint(0, vocab, (n,), generator=g, device="cuda").tolist() for n in (600, 75)]
    last = server.prompt([prompts[b // samples] if b % samples == 0 else [] for b in range(rows)])
    src = [b - b % samples for b in range(rows)]
    server.fork(src)
    live = torch.ones(rows, dtype=torch.bool, device="cuda")
    out, mean = server.sample(last[src], live, steps, [0, 0, 0, 1, 1, 3, 3], g)
    print(f"{rows} samples of {len(prompts)} prompts, {mean:.2f} tokens a step from trees of 7; status {server.status()}")
    server.fork([0, -1, -1, -1, 4, -1, -1, -1])              # one sample of each goes on, the pages of the others are free
    held = int((server.pages.refs > 0).sum())
    return server, out, mean, held


if __name__ == "__main__":
    main()
