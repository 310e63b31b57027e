"""A small language model with random weights whose layers are gated-delta layers and softmax attention layers over a 4-bit KV cache.

  python examples/hybrid_layers.py

It takes a ragged batch of prompts in chunks, generates tokens one at a time, and, with attention layers only, several at a time by
verifying a tree of drafts: one call appends and attends to the whole tree, the path that the model itself would have taken is kept,
the other branches are overwritten by the next step. (A recurrent state holds one history, so a stack with gated-delta layers takes
its tokens one at a time.)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_gated_delta_gb300 as P  # noqa: E402

CHUNK = 256


class Stack:
    """`kinds`: "delta" or "attend" for each layer. All caches share one page table and one vector of lengths."""

    def __init__(self, kinds, batch, max_tokens, vocab=512, heads=8, kv_heads=2, d=128, bits=4, page=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kinds, self.B, self.heads, self.kv_heads, self.d, self.page = kinds, batch, heads, kv_heads, d, page
        self.dm = heads * d
        w = lambda o, i: (torch.randn(o, i, generator=g, device="cuda") * i ** -0.5).bfloat16()
        self.embed, self.unembed = w(vocab, self.dm) * self.dm ** 0.5, w(vocab, self.dm)
        self.rope = P.PaceRope(d, max_tokens + CHUNK)
        self.cols = (max_tokens + CHUNK + page - 1) // page
        self.table = torch.randperm(batch * self.cols, generator=g, device="cuda").int().view(batch, self.cols)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.layers = []
        for kind in kinds:
            if kind == "attend":
                cfg = P.make_kv_config(heads, kv_heads, d, batch * self.cols, batch, bits=bits, page_tokens=page, max_new=CHUNK)
                self.layers.append((P.PaceKV(cfg), w((heads + 2 * kv_heads) * d, self.dm), w(self.dm, self.dm)))
            else:
                state = P.PaceState(P.make_config(heads, d, batch), batch)
                self.layers.append((state, w(3 * self.dm, self.dm), w(self.dm, self.dm), w(2 * heads, self.dm)))

    def attend(self, layer, x, n_new, positions, mask):
        kv, wqkv, wo = layer
        B, T, _ = x.shape
        q, k, v = (x @ wqkv.t()).view(B, T, -1, self.d).split([self.heads, self.kv_heads, self.kv_heads], 2)
        qr, o = torch.empty(2, B, T, self.heads, self.d, dtype=x.dtype, device=x.device)
        kv.append(q, k, v, self.lens, self.table, rope=self.rope, positions=positions, n_new=n_new, q_out=qr)
        kv.attend(qr, o, self.lens, self.table, mask=mask, n_new=n_new)
        return o.flatten(2) @ wo.t()

    def delta(self, layer, x):
        state, wqkv, wo, wab = layer
        B, T, _ = x.shape
        q, k, v = (x @ wqkv.t()).view(B, T, 3, self.heads, self.d).permute(2, 0, 3, 1, 4).contiguous()
        q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(x.dtype) for t in (q, k))
        a, beta = torch.sigmoid((x @ wab.t()).float()).view(B, T, 2, self.heads).permute(2, 0, 3, 1).contiguous()
        a = 1 - 0.1 * a
        o = torch.empty_like(v)
        if T == 1:
            state.decode_step(*(t.squeeze(2) for t in (q, k, v)), a[..., 0].contiguous(), beta[..., 0].contiguous(), o.squeeze(2))
        else:
            state.prefill_chunk(q, k, v, a, beta, o)
        return o.transpose(1, 2).flatten(2) @ wo.t()

    def forward(self, tokens, n_new=None, positions=None, mask=None):
        """Logits [B, T, vocab] of new tokens [B, T], written to every layer; lens is the caller's to advance."""
        x = self.embed[tokens.long()]
        for kind, layer in zip(self.kinds, self.layers):
            h = torch.nn.functional.normalize(x.float(), dim=-1).mul(self.dm ** 0.5).to(x.dtype)
            x = x + (self.attend(layer, h, n_new, positions, mask) if kind == "attend" else self.delta(layer, h))
        return (x @ self.unembed.t()).float()

    def prompt(self, tokens, n=None):
        """Takes prompts [B, T] of n[b] tokens (all T without n) in chunks; returns the token that follows each."""
        last = torch.zeros(self.B, dtype=torch.int64, device="cuda")
        for t0 in range(0, tokens.shape[1], CHUNK):
            part = tokens[:, t0:t0 + CHUNK]
            T = part.shape[1]
            new = torch.full((self.B,), T, dtype=torch.int32, device="cuda") if n is None else (n - t0).clamp(0, T).int()
            best = self.forward(part, None if n is None else new).argmax(-1)
            at = (new.long() - 1).clamp(min=0)
            last = torch.where(new > 0, best.gather(1, at[:, None])[:, 0], last)
            self.lens += new
        return last

    def generate(self, token, steps):
        """Greedy, one token a step: [B, steps]."""
        out = []
        for _ in range(steps):
            token = self.forward(token[:, None])[:, 0].argmax(-1)
            self.lens += 1
            out.append(token)
        return torch.stack(out, 1)

    def generate_drafted(self, token, steps, draft, parents):
        """Greedy, verifying a tree of drafts a step. draft(token [B]) -> tokens [B, N] of a tree whose node 0 is `token` itself and
        whose node i > 0 has the parent parents[i] < i. Returns [B, steps] and the mean number of tokens a step."""
        if "delta" in self.kinds:
            raise ValueError("a recurrent state holds one history: drafts need attention layers only")
        N, dev = len(parents), self.lens.device
        see = torch.zeros(N, N, dtype=torch.bool)
        depth = torch.zeros(N, dtype=torch.int64)
        for i in range(N):
            if i:
                see[i], depth[i] = see[parents[i]], depth[parents[i]] + 1
            see[i, i] = True
        words = torch.zeros(N, (N + 31) // 32, dtype=torch.int64)
        for j in range(N):
            words[:, j // 32] |= see[:, j].long() << (j % 32)
        mask = words.to(torch.uint32).view(torch.int32).to(dev).expand(self.B, -1, -1).contiguous()
        depth, parent = depth.int().to(dev), torch.tensor(parents, device=dev)
        deepest = int(depth.max())
        out, counts, used = [[] for _ in range(self.B)], 0, 0
        while min(map(len, out)) < steps:
            tree = draft(token)
            best = self.forward(tree, positions=self.lens[:, None] + depth, mask=mask).argmax(-1)    # what follows each node
            # a node is accepted where its parent is and predicts it; of the accepted nodes of one depth at most one is
            ok = torch.zeros(self.B, N, dtype=torch.bool, device=dev)
            ok[:, 0] = True
            for i in range(1, N):
                same = (tree[:, 1:i] == tree[:, i:i + 1]) & (parent[1:i] == parent[i])               # (a second branch with the same token)
                ok[:, i] = ok[:, parents[i]] & (best[:, parents[i]] == tree[:, i]) & ~same.any(1)
            n_keep = ok.sum(1).int()
            idx = torch.arange(N, device=dev).expand(self.B, N).masked_fill(~ok, N).sort(1).values[:, :deepest + 1]
            idx = torch.where(idx == N, idx[:, :1], idx).int().contiguous()
            for kv, *_ in self.layers:
                kv.keep(self.lens, self.table, idx, n_keep)
            self.lens += n_keep
            tail = idx.gather(1, (n_keep.long() - 1)[:, None]).long()
            token = best.gather(1, tail)[:, 0]
            follow = best.gather(1, idx.long()).tolist()
            for b, n in enumerate(n_keep.tolist()):
                out[b] += follow[b][:n]
                counts += n
            used += self.B
        return torch.tensor([o[:steps] for o in out], device=dev), counts / used

    def status(self):
        return [layer[0].status() for kind, layer in zip(self.kinds, self.layers) if kind == "attend"]


def main():
    B, vocab = 4, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = torch.randint(0, vocab, (B, 600), generator=g, device="cuda")
    n = torch.tensor([600, 411, 256, 7], device="cuda")

    model = Stack(["delta", "delta", "attend"], B, 1024)
    first = model.prompt(prompts[:, :512])                  # (the gated-delta prefill takes whole chunks: equal prompts)
    tokens = model.generate(first, 32)
    print("hybrid: first tokens", tokens[:, :6].tolist())

    plain = Stack(["attend"], B, 1024)
    first = plain.prompt(prompts, n)
    want = plain.generate(first, 64)
    # drafts: of two guesses a level one is right three times in four (an oracle stands in for a draft model here)
    tree = Stack(["attend"], B, 1024)
    first = tree.prompt(prompts, n)
    parents = [0, 0, 0, 1, 1, 2, 2, 3, 3]
    follows = {}
    for b in range(B):
        seq = [int(first[b])] + want[b].tolist()
        follows.update({(b, i): seq[i:i + 4] for i in range(len(seq))})
    where = [0] * B

    def draft(token):
        rows = []
        for b in range(B):
            where[b] = int(tree.lens[b] - n[b])
            path = (follows.get((b, where[b])) or [int(token[b])]) + [0] * 4
            rnd = torch.randint(0, vocab, (9,), generator=g, device="cuda").tolist()
            good = [path[0], path[1], rnd[2], path[2], rnd[4], rnd[5], rnd[6], path[3], rnd[8]]
            if rnd[0] % 4 == 0:
                good[3] = rnd[3]
            rows.append([int(token[b])] + good[1:])
        return torch.tensor(rows, device="cuda")

    got, mean = tree.generate_drafted(first, 64, draft, parents)
    agree = (got == want).float().mean().item()
    print(f"attention: trees of {len(parents)} drafts give {mean:.2f} tokens a step, {100 * agree:.1f}% of them as one at a time; "
          f"status {plain.status()} {tree.status()}")
    return model, plain, tree, want, got, mean


if __name__ == "__main__":
    main()
