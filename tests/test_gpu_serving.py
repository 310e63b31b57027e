"""The operators of include/pace_serve.h together, as a serving loop uses them: prompts through a cache and recurrent states, rows forked into
samples, trees of drafts appended, attended to, carried through the states and verified, accepted paths kept, pages taken, copied, given
back and compacted. Keys, values and gates are functions of the token alone, so that whatever a row went through, its cache holds the codes
of its tokens and its state what the rule gives them one by one.

Tolerances: codes are equal; states and outputs as in test_gpu_delta.py and (attention) within half a step of bf16 and the 11 bits of its weights
and queries: 2^-8 of the value and 2^-9 of the rms.
"""
import numpy as np
import pytest

import kv_testlib as K
import serve_testlib as T
from pace_testlib import ensure_built

pytestmark = pytest.mark.gpu
VOCAB, H, HKV, D, PAGE = 40, 4, 2, 64, 32


@pytest.fixture(scope="module")
def P():
    ensure_built()
    import bit_gated_delta_gb300 as P
    return P


class Loop:
    def __init__(self, P, rows, cols, seed):
        import torch
        self.P, self.torch, self.rows = P, torch, rows
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)
        unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).bfloat16()
        self.q, self.k, self.v = unit(r(VOCAB, HKV, D)), unit(r(VOCAB, HKV, D)), r(VOCAB, H, D).bfloat16()
        self.qa, self.va = r(VOCAB, H, D).bfloat16(), r(VOCAB, HKV, D).bfloat16()
        self.a, self.beta = 0.9 + 0.1 * torch.rand(VOCAB, H, generator=g), torch.rand(VOCAB, H, generator=g)
        self.n_pages = rows * cols
        self.kv = P.PaceKV(P.make_kv_config(H, HKV, D, self.n_pages, rows, bits=8, page_tokens=PAGE))
        self.delta = P.PaceDelta(P.make_delta_config(H, D, rows, key_heads=HKV))
        self.pages = P.PacePages(self.n_pages, PAGE, rows)
        self.table = torch.full((rows, cols), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.history = [[] for _ in range(rows)]
        self.dev = {n: getattr(self, n).cuda() for n in ("q", "k", "v", "qa", "va", "a", "beta")}

    def ints(self, x):
        return self.torch.tensor(np.asarray(x), dtype=self.torch.int32, device="cuda")

    def take(self, n):
        fits = self.torch.empty(self.rows, dtype=self.torch.int32, device="cuda")
        self.pages.take(self.table, self.lens, n, fits)
        self.kv.copy_pages(self.pages)
        assert bool(fits.all())

    def layers(self, tokens, n, mask=None):
        """Appends and attends, and the outputs of both layers; a tree leaves the states alone."""
        d, t = self.dev, tokens.long()
        oa, o = (self.torch.empty(*tokens.shape, H, D, dtype=self.torch.bfloat16, device="cuda") for _ in range(2))
        self.kv.append(None, d["k"][t], d["va"][t], self.lens, self.table, n_new=n)
        self.kv.attend(d["qa"][t], oa, self.lens, self.table, mask=mask, n_new=n)
        args = [d[x][t] for x in ("q", "k", "v", "a", "beta")]
        if mask is None:
            self.delta.chunk(*args, o, lens=self.lens, n_new=n)
        else:
            self.delta.draft(*args, o, n_new=n, mask=mask)
        return oa, o, args

    def prompt(self, prompts):
        n = [len(p) for p in prompts]
        tokens = np.zeros((self.rows, max(n)), np.int32)
        for b, p in enumerate(prompts):
            tokens[b, :len(p)] = p
            self.history[b] += list(p)
        n = self.ints(n)
        self.take(n)
        self.layers(self.ints(tokens), n)
        self.lens += n

    def fork(self, src):
        self.pages.select(self.table, self.lens, self.ints(src))
        pick = self.torch.tensor([max(s, 0) for s in src], device="cuda")
        self.delta.states.copy_(self.delta.states[pick])
        self.history = [list(self.history[s]) if s >= 0 else [] for s in src]

    def drafted(self, rng, N):
        """One step of trees of N nodes, node 0 the last token that is not in the caches yet."""
        torch, B = self.torch, self.rows
        parents = np.zeros((B, N), int)
        see = np.zeros((B, N, N), bool)
        for b in range(B):
            for i in range(N):
                parents[b, i] = max(0, i - 1 - rng.integers(0, 3)) if i else -1
                see[b, i] = see[b, parents[b, i]] if i else False
                see[b, i, i] = True
        p = torch.softmax(torch.tensor(rng.normal(size=(B, N, VOCAB)) * 2), -1).float()
        q = torch.softmax(torch.log(p) + torch.tensor(rng.normal(size=(B, N, VOCAB)) * 0.5), -1).float()
        tokens = np.zeros((B, N), np.int32)
        for b in range(B):
            tokens[b, 0] = rng.integers(0, VOCAB)
            for i in range(1, N):
                w = q[b, parents[b, i]].double().numpy()
                tokens[b, i] = rng.choice(VOCAB, p=w / w.sum())
        live = [len(h) > 0 for h in self.history]
        n = self.ints([N if x else 0 for x in live])
        u = torch.tensor(rng.random((B, N)), dtype=torch.float32)
        bits = (see[..., None, :] * (1 << np.arange(N, dtype=np.uint64))).sum(-1).astype(np.uint32)
        mask = torch.from_numpy(bits.view(np.int32)).cuda()
        self.take(n)
        oa, o, args = self.layers(self.ints(tokens), n, mask)
        idx = torch.empty(B, N, dtype=torch.int32, device="cuda")
        n_keep, nxt = torch.empty(2, B, dtype=torch.int32, device="cuda")
        self.P.pace_verify(self.ints(tokens), p.cuda(), q.cuda(), u.cuda(), idx, n_keep, nxt, mask=mask, n_new=n)
        self.check(tokens, see, live, oa, o)
        self.kv.keep(self.lens, self.table, idx, n_keep)
        self.delta.keep(*args[1:], idx, n_keep)
        self.lens += n_keep
        self.pages.select(self.table, self.lens)             # pages of tokens that were not kept go back
        for b in range(B):
            if live[b]:
                path, _ = T.verify(tokens[b], p[b].numpy(), q[b].numpy(), u[b].numpy(), parents[b])
                assert idx[b, :n_keep[b]].tolist() == path
                self.history[b] += [int(tokens[b, i]) for i in path]
            else:
                assert int(n_keep[b]) == 0 and int(nxt[b]) == -1

    def state(self, b):
        f = lambda x: x.float().numpy().astype(np.float64)
        S = np.zeros((H, D, D))
        k, v, a, beta = f(self.k), f(self.v), f(self.a), f(self.beta)
        for t in self.history[b]:
            for h in range(H):
                S[h] = T.rule(S[h], k[t, h // (H // HKV)], v[t, h], a[t, h], beta[t, h])
        return S

    def check(self, tokens, see, live, oa, o):
        """Outputs of a tree against the rule and softmax over the held values."""
        f = lambda x: x.float().cpu().numpy().astype(np.float64)
        held_k, held_v = K.held(self.k.float().numpy(), 8), K.held(self.va.float().numpy(), 8)
        for b in range(self.rows):
            t = tokens[b]
            if not live[b]:
                assert not oa[b].any() and not o[b].any()
                continue
            S = self.state(b)
            for h in range(H):
                want = T.draft(S[h], f(self.q)[t, h // 2], f(self.k)[t, h // 2], f(self.v)[t, h], f(self.a)[t, h], f(self.beta)[t, h], see[b])
                rms = np.sqrt((want ** 2).mean())
                assert (np.abs(f(o[b, :, h]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * rms).all()
                past = np.array(self.history[b], int)
                for i in range(len(t)):
                    slots = np.concatenate([past, t[see[b, i]]])
                    w = np.exp(f(self.qa)[t[i], h] @ held_k[slots, h // 2].T * D ** -0.5)
                    y = w @ held_v[slots, h // 2] / w.sum()
                    assert (np.abs(f(oa[b, i, h]) - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -9 * np.sqrt((y ** 2).mean())).all()

    def settled(self):
        """Caches, states, counts of pages and lengths are those of the rows' tokens."""
        torch = self.torch
        n = max(map(len, self.history))
        k, v = torch.empty(2, self.rows, n, HKV, D, dtype=torch.bfloat16, device="cuda")
        self.kv.read(k, v, self.table, end=self.lens)
        refs = np.zeros(self.n_pages, int)
        for b, past in enumerate(self.history):
            assert int(self.lens[b]) == len(past)
            for x, want in ((k, self.k), (v, self.va)):
                held = torch.from_numpy(K.held(want.float().numpy(), 8)).bfloat16()
                assert torch.equal(x[b, :len(past)].cpu(), held[past]) and not x[b, len(past):].any()
            cells = self.table[b].tolist()
            cover = -(-len(past) // PAGE)
            assert all(c >= 0 for c in cells[:cover]) and all(c == -1 for c in cells[cover:])
            for c in cells[:cover]:
                refs[c] += 1
            if past:
                want = self.state(b)
                got = self.delta.states[b].double().cpu().numpy()
                assert (np.abs(got - want) <= 2.0 ** -16 * np.sqrt((want ** 2).mean())).all()
        assert np.array_equal(self.pages.refs.cpu().numpy(), refs)
        assert self.kv.status() == self.delta.status() == self.pages.status() == 0


@pytest.mark.parametrize("seed", [0, 1])
def test_a_serving_loop(P, seed):
    rng = np.random.default_rng(seed)
    x = Loop(P, rows=6, cols=9, seed=seed)
    x.prompt([rng.integers(0, VOCAB, n) for n in (70, 0, 0, 33, 1, 0)])
    x.settled()
    x.fork([0, 0, 0, 3, 4, -1])                  # three samples of the first prompt
    for N in (5, 9, 2):
        x.drafted(rng, N)
        x.settled()
    x.fork([1, 1, 3, 0, -1, 4])                  # the rows change places, one goes on twice, one is given up
    x.drafted(rng, 12)
    x.settled()
    x.pages.compact(x.table)
    x.kv.copy_pages(x.pages)
    used = int((x.pages.refs > 0).sum())
    assert int(x.table.max()) == used - 1
    x.settled()
    x.drafted(rng, 7)
    x.settled()
