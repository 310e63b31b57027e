"""Verification of drafts against its statement in 64 bits: whole numbers, equal everywhere. (The kernel's sums are exact to 2^-46 a token, so
that a draw could differ only where u_0 falls within about 2^-38 of a border; the seeds here do not.)"""
import numpy as np
import pytest

import serve_testlib as T
from pace_testlib import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    ensure_built()
    import bit_gated_delta_gb300 as P
    return P


def tree(rng, N, chain):
    parents = np.arange(-1, N - 1)
    if not chain:
        for i in range(1, N):
            parents[i] = max(0, i - 1 - rng.integers(0, 5))
    see = np.eye(N, dtype=bool)
    for i in range(1, N):
        see[i] |= see[parents[i]]
    return parents, see


def words(torch, see):
    n = see.shape[-1]
    W = (n + 31) // 32
    bits = np.zeros(see.shape[:-1] + (W * 32,), np.uint64)
    bits[..., :n] = see
    w = (bits.reshape(see.shape[:-1] + (W, 32)) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return torch.from_numpy(w.view(np.int32)).cuda()


def softmax(torch, x, dt):
    return torch.softmax(x, -1).to(dt).cuda()


def call(P, torch, tokens, p, q, u, mask=None, n_new=None):
    B, N = tokens.shape
    idx = torch.full((B, N), -7, dtype=torch.int32, device="cuda")
    n_keep, nxt = torch.full((2, B), -7, dtype=torch.int32, device="cuda")
    P.pace_verify(tokens, p, q, u, idx, n_keep, nxt, mask=mask, n_new=n_new)
    return idx.cpu().numpy(), n_keep.cpu().numpy(), nxt.cpu().numpy()


def check(P, torch, tokens, p, q, u, parents, mask=None, n_new=None):
    B, N = tokens.shape
    idx, n_keep, nxt = call(P, torch, tokens, p, q, u, mask, n_new)
    tok, un = tokens.cpu().numpy(), u.cpu().numpy()
    for b in range(B):
        n = N if n_new is None else min(max(int(n_new[b]), 0), N)
        if n == 0:
            assert n_keep[b] == 0 and nxt[b] == -1 and not idx[b].any()
            continue
        path, want = T.verify(tok[b, :n], p[b, :n].float().cpu().numpy(), None if q is None else q[b, :n].float().cpu().numpy(), un[b], parents[b])
        assert idx[b, :n_keep[b]].tolist() == path and nxt[b] == want
        assert (idx[b, n_keep[b]:] == path[-1]).all()
    return n_keep, nxt


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("named", [False, True])
@pytest.mark.parametrize("B,N,V,chain", [(1, 1, 1, True), (3, 2, 7, True), (2, 5, 33, False), (4, 9, 2049, True), (5, 25, 4097, False),
                                         (2, 70, 5000, False), (3, 256, 300, False), (40, 6, 20001, True), (90, 4, 9000, False),
                                         (200, 3, 4500, True), (400, 2, 1000, True), (1, 4, 262144, True)])
def test_verification(P, B, N, V, chain, named, dtype):
    import torch
    dt = getattr(torch, dtype)
    g = torch.Generator().manual_seed(B * 1000 + N)
    rng = np.random.default_rng(V)
    logits = torch.randn(B, N, V, generator=g) * 2
    p = softmax(torch, logits, dt)
    q = softmax(torch, logits + torch.randn(B, N, V, generator=g) * 0.8, dt)
    trees = [tree(rng, N, chain) for _ in range(B)]
    parents = np.stack([t[0] for t in trees])
    draft = q.float().cpu()
    tok = torch.zeros(B, N, dtype=torch.int32)
    for b in range(B):
        for i in range(1, N):
            row = draft[b, parents[b, i]]
            tok[b, i] = int(torch.multinomial(row, 1, generator=g)) if not named else int(row.argmax()) if i % 2 else int(torch.randint(0, V, (1,), generator=g))
    u = torch.rand(B, N, generator=g).cuda()
    mask = None if chain else words(torch, np.stack([t[1] for t in trees]))
    n_new = torch.tensor([max(0, N - b) for b in range(B)], dtype=torch.int32, device="cuda") if B in (3, 5) else None
    kept, _ = check(P, torch, tok.cuda(), p, None if named else q, u, parents, mask, n_new)
    if N > 2 and not named and n_new is None and B * N > 20:
        assert kept.max() > 1


def test_refused_siblings_share_what_is_left(P):
    """Several drafts of one node, refused one after the other: each sum is that of what the ones before left."""
    import torch
    B, N, V = 64, 6, 1500
    g = torch.Generator().manual_seed(3)
    p = softmax(torch, torch.randn(B, N, V, generator=g) * 3, torch.float32)
    q = softmax(torch, torch.randn(B, N, V, generator=g) * 3, torch.float32)
    parents = np.tile(np.array([-1, 0, 0, 0, 0, 0]), (B, 1))
    see = np.eye(N, dtype=bool)
    see[1:, 0] = True
    tok = torch.multinomial(q[:, 0].cpu(), N, replacement=True, generator=g).int().cuda()
    tok[:, 4] = tok[:, 2]                       # the same token twice
    u = torch.rand(B, N, generator=g).cuda()
    mask = words(torch, np.tile(see, (B, 1, 1)))
    kept, _ = check(P, torch, tok, p, q, u, parents, mask)
    assert 0 < (kept == 1).sum() < B
    check(P, torch, tok, p, None, u, parents, mask)


def test_tokens_are_distributed_as_the_targets(P):
    """One draft from q, kept or replaced: over many random numbers the next token has the target's frequencies. 65,536 trials: a
    frequency f is off by sqrt(f (1 - f) / 65536) < 0.002; five of those."""
    import torch
    V, B = 6, 1024
    p = torch.tensor([0.30, 0.05, 0.25, 0.10, 0.0, 0.30])
    q = torch.tensor([0.05, 0.45, 0.10, 0.10, 0.20, 0.10])
    g = torch.Generator().manual_seed(9)
    count = torch.zeros(V)
    pp = p.expand(B, 2, V).contiguous().cuda()
    qq = q.expand(B, 2, V).contiguous().cuda()
    for _ in range(64):
        tok = torch.multinomial(q, B * 2, replacement=True, generator=g).view(B, 2).int()
        idx, n, nxt = call(P, torch, tok.cuda(), pp, qq, torch.rand(B, 2, generator=g).cuda())
        first = np.where(n == 2, tok[:, 1].numpy(), nxt)
        count += torch.bincount(torch.from_numpy(first.astype(np.int64)), minlength=V)
    assert (count / count.sum() - p).abs().max() < 0.01


def test_random_numbers_at_their_ends(P):
    import torch
    V = 3000
    p = torch.zeros(3, 2, V, device="cuda")
    p[:, :, 5], p[:, :, 2990] = 0.25, 0.75
    tok = torch.tensor([[0, 2990], [0, 2990], [0, 7]], dtype=torch.int32, device="cuda")
    last = float(np.nextafter(np.float32(1), np.float32(0)))
    for u, want, kept in ((0.0, [5, 5, 5], [2, 2, 1]), (last, [2990, 5, 2990], [1, 1, 1]), (1.0, [5, 5, 2990], [1, 1, 1])):
        uu = torch.full((3, 2), u, device="cuda")
        idx, n, nxt = call(P, torch, tok, p, None, uu)
        assert n.tolist() == kept
        assert all(x in (5, 2990) for x in nxt.tolist()) and nxt[2] == want[2]


def test_nothing_left_and_nothing_there(P):
    import torch
    V = 100
    p = torch.zeros(5, 2, V, device="cuda")
    p[0, :, 3] = 1.0                             # refused although certain: u is out of range; its own row is drawn from
    p[1] = 0.0                                   # no probability at all
    p[2] = float("nan")
    p[3, :, 4] = float("inf")                    # counts as 1
    p[4, :, 9] = 0.5
    tok = torch.full((5, 2), 3, dtype=torch.int32, device="cuda")
    tok[4, 1] = 100                              # outside the vocabulary
    u = torch.full((5, 2), 1.0, device="cuda")
    u[:, 0] = 0.5
    for q in (None, p.nan_to_num(0.0, 1.0).contiguous()):
        idx, n, nxt = call(P, torch, tok, p, q, u)
        assert n.tolist() == [1] * 5 and nxt.tolist() == [3, -1, -1, 4, 9]


def test_nodes_that_hang_nowhere_are_not_kept(P):
    import torch
    V, N = 50, 4
    p = torch.full((1, N, V), 1 / V, device="cuda")
    tok = torch.zeros(1, N, dtype=torch.int32, device="cuda")
    u = torch.zeros(1, N, device="cuda")
    see = np.eye(N, dtype=bool)[None].copy()
    see[0, 3, 0] = True
    idx, n, nxt = call(P, torch, tok, p, None, u, words(torch, see))
    assert idx[0, :n[0]].tolist() == [0, 3]


def test_rows_of_any_strides(P):
    """Vocabularies cut out of wider rows, nodes and batches in another order."""
    import torch
    B, N, V = 3, 5, 1001
    g = torch.Generator().manual_seed(1)
    for dt in (torch.float32, torch.bfloat16):
        wide = softmax(torch, torch.randn(N, B, V + 37, generator=g) * 2, dt)
        other = softmax(torch, torch.randn(B, N, V + 3, generator=g) * 2, dt)
        p, q = wide[:, :, 3:3 + V].transpose(0, 1), other[:, :, 1:1 + V]
        tok = torch.randint(0, V, (B, N), generator=g, dtype=torch.int32).cuda()
        u = torch.rand(B, N, generator=g).cuda() * 0.3
        check(P, torch, tok, p, q, u, np.tile(np.arange(-1, N - 1), (B, 1)))


def test_offsets_past_32_bits(P):
    """A row that lies more than 2^32 bytes into the tensor."""
    import torch
    V, N = 70000, 40
    p = torch.zeros(400, N, V, dtype=torch.float32, device="cuda")      # 4.5 GB
    p[399, :, 69999] = 1.0
    p[0, :, 3] = 1.0
    tok = torch.zeros(400, N, dtype=torch.int32, device="cuda")
    tok[399] = 69999
    idx, n, nxt = call(P, torch, tok, p, None, torch.full((400, N), 0.5, device="cuda"))
    assert n[399] == N and nxt[399] == 69999 and n[0] == 1 and nxt[0] == 3 and nxt[1] == -1


def test_same_tokens_on_any_stream_and_in_a_graph(P):
    import torch
    B, N, V = 6, 5, 30000
    g = torch.Generator().manual_seed(2)
    p, q = (softmax(torch, torch.randn(B, N, V, generator=g) * 2, torch.float32) for _ in range(2))
    tok, u = torch.randint(0, V, (B, N), generator=g, dtype=torch.int32).cuda(), torch.rand(B, N, generator=g).cuda()
    want = call(P, torch, tok, p, q, u)
    idx, out = torch.zeros(B, N, dtype=torch.int32, device="cuda"), torch.zeros(2, B, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    P.pace_verify(tok, p, q, u, idx, out[0], out[1], stream=side)
    side.synchronize()
    assert np.array_equal(idx.cpu(), want[0]) and np.array_equal(out.cpu(), want[1:])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.pace_verify(tok, p, q, u, idx, out[0], out[1])
    idx.zero_(), out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(idx.cpu(), want[0]) and np.array_equal(out.cpu(), want[1:])


def test_refusals(P):
    import torch
    p = torch.zeros(2, 3, 10, device="cuda")
    i, u = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, device="cuda")
    one = torch.zeros(2, dtype=torch.int32, device="cuda")
    good = dict(tokens=i, p=p, q=None, u=u, idx=i.clone(), n_keep=one, next=one.clone())
    for bad in (dict(p=p.double()), dict(p=p.transpose(1, 2)), dict(q=p.bfloat16()), dict(u=u.double()), dict(u=u[:, :2]), dict(tokens=i.long()),
                dict(idx=i[:, :2]), dict(n_keep=i), dict(mask=i), dict(p=p[..., ::2]), dict(p=p.cpu())):
        with pytest.raises(ValueError):
            P.pace_verify(**{**good, **bad})
    many = torch.zeros(1, 257, 4, device="cuda")
    with pytest.raises(P.PaceError, match="n_nodes"):
        P.pace_verify(torch.zeros(1, 257, dtype=torch.int32, device="cuda"), many, None, many[..., 0].contiguous(),
                      torch.zeros(1, 257, dtype=torch.int32, device="cuda"), one[:1], one[:1].clone())
