"""Measured cases of the operators that serve drafts and changing sets of sequences: the gated delta rule over fp32 states in
slots (prompts, single tokens, trees of drafts, accepted paths), verification of drafted tokens against the target's
probabilities, and the pages of a cache (shared, taken, given back, compacted, copied).

`own` False computes every pass in plain torch operations; `own` True makes the calls a user of bit_gated_delta_gb300 makes. Both
read the same seeded inputs.

The gated delta rule: S_t = a_t S_{t-1} + k_t u_t^T, u_t = beta_t (v_t - a_t S_{t-1}^T k_t), o_t = S_t^T q_t; in a tree the
state before a token is its parent's.
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 64


def _dt(case):
    return torch.float32 if case["io"] == "f32" else torch.bfloat16


def listed():
    return [
        # one user, one token of a small layer: the latency of a small call
        dict(name="delta_one", kind="chunk", B=1, T=1, H=16, Hk=16, d=64, io="f32", fresh=False),
        # one decode step of 64 sequences, 32 value heads over 16 key heads
        dict(name="delta_decode", kind="chunk", B=64, T=1, H=32, Hk=16, d=128, io="bf16", fresh=False),
        # ragged prompts of a serving batch, from zero states
        dict(name="delta_prompt", kind="chunk", B=16, T=2048, H=32, Hk=16, d=128, io="bf16", fresh=True),
        # two long documents through a 48-head layer, going on from their states
        dict(name="delta_long", kind="chunk", B=2, T=16384, H=48, Hk=48, d=128, io="bf16", fresh=False),
        # odd prompts of a small layer in fp32 (calibration of a quantized state)
        dict(name="delta_calib", kind="chunk", B=4, T=777, H=16, Hk=8, d=64, io="f32", fresh=True),
        # 25 drafts a sequence as a tree, then the accepted path into the states
        dict(name="delta_draft", kind="draft", B=32, T=25, H=32, Hk=16, d=128, io="bf16", tree=True),
        # one sequence, four drafts in a row over a small vocabulary
        dict(name="verify_one", kind="verify", B=1, N=5, V=8192, io="f32", tree=False, drafts="probabilities"),
        # a serving batch with seven drafts in a row over a large vocabulary
        dict(name="verify_batch", kind="verify", B=64, N=8, V=131072, io="f32", tree=False, drafts="probabilities"),
        # trees of 25 nodes whose tokens a draft model named without probabilities
        dict(name="verify_tree", kind="verify", B=16, N=25, V=50001, io="bf16", tree=True, drafts="tokens"),
        # a decode step's bookkeeping: pages for eight drafts of 256 sequences, and the unused ones back
        dict(name="pages_step", kind="pages", B=256, samples=1, new=8, page=32, cols=128, Hkv=1, d=64, bits=4, copy=False),
        # 16 prompts of up to 8k tokens, each gone on with four samples: rows shared, last pages copied, samples given up
        dict(name="pages_fork", kind="pages", B=64, samples=4, new=1, page=64, cols=130, Hkv=8, d=128, bits=8, copy=True),
        # a pool of 8192 pages of which more than a quarter are in use, moved to its front
        dict(name="pages_compact", kind="compact", B=64, page=64, cols=48, n_pages=8192, Hkv=8, d=128, bits=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.7e12 + w["flops"] / 1.0e14


def draw(rng):
    tops = {}
    for c in listed():
        tops[c["kind"]] = max(tops.get(c["kind"], 0.0), _cost(c))
    while True:
        kind = rng.choice(["chunk", "chunk", "chunk", "draft", "verify", "verify", "pages", "compact"])
        if kind in ("chunk", "draft"):
            hk = rng.randint(1, 16)
            case = dict(kind=kind, H=hk * rng.choice([1, 2, 3]), Hk=hk, d=rng.choice([64, 128, 128]),
                        io=rng.choice(["bf16", "bf16", "f32"]))
            if kind == "draft":
                case.update(B=_log_int(rng, 1, 64), T=_log_int(rng, 1, 64), tree=rng.random() < 0.6)
            elif rng.random() < 0.35:
                case.update(B=_log_int(rng, 1, 128), T=rng.choice([1, 1, 2, 3, 5, 9]), fresh=False)
            else:
                case.update(B=_log_int(rng, 1, 32), T=_log_int(rng, 10, 16384), fresh=rng.random() < 0.5)
            if case["B"] * case["T"] * case["H"] > 2 * 16384 * 48:
                continue
        elif kind == "verify":
            tree = rng.random() < 0.5
            case = dict(kind=kind, B=_log_int(rng, 1, 64), N=_log_int(rng, 1, 64) if tree else rng.randint(1, 16),
                        V=_log_int(rng, 500, 200000), io=rng.choice(["f32", "f32", "bf16"]), tree=tree,
                        drafts=rng.choice(["probabilities", "tokens"]))
            if case["B"] * case["N"] * case["V"] > 64 * 8 * 131072:
                continue
        else:
            page, d = rng.choice([32, 64, 128]), rng.choice([64, 128, 256])
            case = dict(kind=kind, page=page, Hkv=rng.choice([1, 2, 3, 4, 8]), d=d, bits=rng.choice([4, 8]))
            if kind == "pages":
                samples = rng.choice([1, 2, 3, 4, 8])
                case.update(B=samples * _log_int(rng, 1, 512 // samples), samples=samples, new=_log_int(rng, 1, 64),
                            cols=_log_int(rng, 3, 200), copy=rng.random() < 0.6)
            else:
                rows = _log_int(rng, 1, 256)
                case.update(B=rows, cols=_log_int(rng, 1, 64), n_pages=0)
                case["n_pages"] = int(rows * case["cols"] * rng.uniform(1.05, 4.0)) + 1
            if _pool_pages(case) * _page_bytes(case) > 4 << 30:
                continue
        if _cost(case) <= tops[kind]:
            return case


# ---- sizes --------------------------------------------------------------------------------------------------------------------
def _counts(case):
    """Ragged token counts of a prompt batch, the same for every seed."""
    B, T = case["B"], case["T"]
    if T < 10:
        return [T] * B
    return [T - int(T * 0.7 * ((b * 0.6180339887498949) % 1.0)) for b in range(B)]


def _page_bytes(case):
    """Codes, bf16 scales and (4 bits) zero points of k and v, groups of 64."""
    ng = case["d"] // 64
    return case["page"] * case["Hkv"] * 2 * (case["d"] * case["bits"] // 8 + 2 * ng + (ng if case["bits"] == 4 else 0))


def _row_lens(case):
    """Lengths of the sequences (one for each group of samples), the same for every seed: half a table or more, room left for new tokens."""
    top = case["cols"] * case["page"] - case.get("new", 0)
    n = case["B"] // case.get("samples", 1)
    return [max(1, top - int(top * 0.5 * ((b * 0.6180339887498949) % 1.0))) for b in range(n)]


def _pool_pages(case):
    if case["kind"] == "compact":
        return case["n_pages"]
    need = sum(-(-n // case["page"]) for n in _row_lens(case))
    return need + case["B"] * (2 + case["new"] // case["page"])


def work(case):
    kind = case["kind"]
    if kind in ("chunk", "draft"):
        B, H, Hk, d = case["B"], case["H"], case["Hk"], case["d"]
        es = 4 if case["io"] == "f32" else 2
        n = sum(_counts(case)) if kind == "chunk" else B * case["T"]
        row = es * (2 * Hk * d + 2 * H * d) + 8 * H
        if kind == "chunk":
            return {"bytes": n * row + B * H * d * d * 4 * (1 if case["fresh"] else 2), "flops": n * H * 6 * d * d}
        path = B * max(1, case["T"] // 4)
        return {"bytes": n * row + B * H * d * d * 4 * 2 + path * (es * (Hk + H) * d + 8 * H),
                "flops": n * H * 4 * d * d + path * H * 4 * d * d}
    if kind == "verify":
        es = 4 if case["io"] == "f32" else 2
        rows = case["B"] * case["V"] * es * (2 if case["drafts"] == "probabilities" else 1)
        return {"bytes": rows + case["B"] * case["N"] * 24, "flops": 3 * case["B"] * case["V"]}
    if kind == "pages":
        cells = case["B"] * case["cols"]
        bytes_ = 4 * (2 * cells + 2 * case["B"] * 4 + 3 * _pool_pages(case))
        if case["copy"]:
            part = sum(n % case["page"] != 0 for n in _row_lens(case))
            bytes_ += 2 * _page_bytes(case) * part * (case["samples"] - 1)
        return {"bytes": bytes_, "flops": 0}
    used = sum(-(-n // case["page"]) for n in _row_lens(case))
    moved = used * (case["n_pages"] - used) // case["n_pages"]
    return {"bytes": 2 * _page_bytes(case) * moved + 4 * (2 * case["n_pages"] + 2 * case["B"] * case["cols"]), "flops": 0}


# ---- inputs ---------------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _tree(B, N, tree, g):
    """parents [B, N] of N nodes (node 0 is a root; a chain, or a node hangs from one of the four before it), and the ancestors
    [B, N, N] of each, itself among them."""
    i = torch.arange(N, device=DEV)
    back = (torch.rand(B, N, generator=g, device=DEV) * 4).long() if tree else torch.zeros(B, N, dtype=torch.long, device=DEV)
    parents = (i - 1 - back).clamp(min=0)
    anc = torch.eye(N, dtype=torch.bool, device=DEV).repeat(B, 1, 1)
    for t in range(1, N):
        anc[:, t] |= torch.gather(anc, 1, parents[:, t, None, None].expand(B, 1, N))[:, 0]
    return parents, anc


def _words(anc):
    """Ancestor bits as 32-bit words, [B, N, ceil(N / 32)]."""
    B, N, _ = anc.shape
    W = (N + 31) // 32
    bits = torch.zeros(B, N, W * 32, dtype=torch.int64, device=DEV)
    bits[..., :N] = anc
    words = (bits.view(B, N, W, 32) << torch.arange(32, device=DEV)).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()


def _delta_inputs(case, g):
    """Unit keys and queries, values with a few larger channels, slow decays, states of some earlier context, in slots of any order."""
    B, T, H, Hk, d, dt = case["B"], case["T"], case["H"], case["Hk"], case["d"], _dt(case)

    def unit(h):
        x = torch.randn(B, T, h, d, generator=g, device=DEV)
        return (x / x.square().sum(-1, keepdim=True).sqrt()).to(dt)

    inp = dict(q=unit(Hk), k=unit(Hk))
    v = torch.randn(B, T, H, d, generator=g, device=DEV)
    big = torch.ones(H, d, device=DEV).scatter_(1, torch.randint(0, d, (H, 4), generator=g, device=DEV), 8.0)
    inp["v"] = (v * big).to(dt)
    inp["a"] = 0.95 + 0.0499 * torch.rand(B, T, H, generator=g, device=DEV)
    inp["beta"] = 1 / (1 + torch.exp(-torch.randn(B, T, H, generator=g, device=DEV)))
    slots = B + B // 4
    inp["states"] = torch.randn(slots, H, d, d, generator=g, device=DEV) * 0.3
    inp["slots"] = torch.randperm(slots, generator=g, device=DEV)[:B].int()
    inp["n_new"] = inp["lens"] = inp["mask"] = None
    if case["kind"] == "chunk":
        n = _counts(case)
        if min(n) < T:
            inp["n_new"] = torch.tensor(n, dtype=torch.int32, device=DEV)
        if case["fresh"]:
            inp["lens"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        return inp
    inp["parents"], inp["anc"] = _tree(B, T, case["tree"], g)
    inp["mask"] = _words(inp["anc"]) if case["tree"] else None
    # the path from the root to some node
    leaf = torch.randint(0, T, (B,), generator=g, device=DEV)
    path = inp["anc"][torch.arange(B, device=DEV), leaf]
    inp["n_keep"] = path.sum(1).int()
    order = torch.where(path, torch.arange(T, device=DEV), T).sort(1).values
    inp["idx"] = torch.where(order == T, order[:, :1], order).int()
    return inp


def _verify_inputs(case, g):
    """Probabilities of a target and of a draft model near it; the drafts come from the draft model."""
    B, N, V, dt = case["B"], case["N"], case["V"], _dt(case)
    inp = {}
    parents, anc = _tree(B, N, case["tree"], g)
    inp["parents"], inp["mask"] = parents, _words(anc) if case["tree"] else None
    logits = torch.randn(B, N, V, generator=g, device=DEV) * 2.5
    inp["p"] = torch.softmax(logits, -1).to(dt)
    logits += torch.randn(B, N, V, generator=g, device=DEV) * 0.7
    draft = torch.softmax(logits, -1).to(dt)
    del logits
    if case["drafts"] == "probabilities":
        cum = draft.float().cumsum(-1)
        cum = cum / cum[..., -1:]
        at = torch.gather(cum, 1, parents[..., None].expand(B, N, V))
        tok = torch.searchsorted(at, torch.rand(B, N, 1, generator=g, device=DEV))[..., 0]
        inp["q"] = draft
    else:                                    # the likeliest tokens, one for each child
        rank = (parents[:, :, None] == parents[:, None, :]).tril(-1).sum(-1).clamp(max=min(4, V - 1))
        top = draft.float().topk(min(5, V), -1).indices
        tok = torch.gather(torch.gather(top, 1, parents[..., None].expand(B, N, top.shape[-1])), 2, rank[..., None])[..., 0]
        inp["q"] = None
    inp["tokens"] = tok.clamp(max=V - 1).int()
    inp["u"] = torch.rand(B, N, generator=g, device=DEV)
    return inp


def _pages_inputs(case, g):
    """Prompts' pages dealt in any order; the rows of their further samples are still empty."""
    B, P, C, n_pages = case["B"], case["page"], case["cols"], _pool_pages(case)
    samples, lens = case.get("samples", 1), _row_lens(case)
    table = torch.full((B, C), -1, dtype=torch.int32, device=DEV)
    row_len = torch.zeros(B, dtype=torch.int32, device=DEV)
    first = torch.arange(0, B, samples, device=DEV)
    row_len[first] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    held = torch.arange(C, device=DEV)[None] < ((row_len + P - 1) // P)[:, None]
    order = torch.randperm(n_pages, generator=g, device=DEV).int()
    table[held] = order[:int(held.sum())]
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    refs[table[held].long()] = 1
    inp = dict(table=table, lens=row_len, refs=refs, n_pages=n_pages)
    i = torch.arange(B, device=DEV)
    inp["fork"] = (i - i % samples).int()
    inp["back"] = torch.where(i % samples == 0, i, -1).int()
    if "new" in case:
        inp["n_new"] = torch.full((B,), case["new"], dtype=torch.int32, device=DEV)
    if case.get("copy", True):
        inp["pool"] = torch.randint(0, 256, (n_pages, _page_bytes(case)), generator=g, device=DEV, dtype=torch.uint8)
    return inp


def _inputs(case, seed):
    g = _gen(seed)
    if case["kind"] in ("chunk", "draft"):
        return _delta_inputs(case, g)
    return _verify_inputs(case, g) if case["kind"] == "verify" else _pages_inputs(case, g)


# ---- the measured interface ---------------------------------------------------------------------------------------------------
def prepare(case, seed):
    st = dict(case=case, inp=_inputs(case, seed))
    inp, kind = st["inp"], case["kind"]
    if own:
        import bit_gated_delta_gb300 as P
        if kind in ("chunk", "draft"):
            cfg = P.make_delta_config(case["H"], case["d"], inp["states"].shape[0], key_heads=case["Hk"],
                                      io_dtype=P.PACE_IO_F32 if case["io"] == "f32" else P.PACE_IO_BF16)
            st["delta"] = P.PaceDelta(cfg)
            st["delta"].states.copy_(inp.pop("states"))
        elif kind in ("pages", "compact"):
            st["pages"] = P.PacePages(inp["n_pages"], case["page"], case["B"])
            st["pages"].refs.copy_(inp["refs"])
            if "pool" in inp:
                st["kv"] = P.PaceKV(P.make_kv_config(case["Hkv"], case["Hkv"], case["d"], inp["n_pages"], case["B"],
                                                     bits=case["bits"], page_tokens=case["page"]))
                st["kv"].pages().copy_(inp.pop("pool"))
    return st


def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import bit_gated_delta_gb300 as P
    case, inp, kind = st["case"], st["inp"], st["case"]["kind"]
    if kind in ("chunk", "draft"):
        delta, o = st["delta"], torch.empty_like(inp["v"])
        x = [inp[n] for n in ("q", "k", "v", "a", "beta")]
        if kind == "chunk":
            delta.chunk(*x, o, slots=inp["slots"], lens=inp["lens"], n_new=inp["n_new"])
        else:
            delta.draft(*x, o, slots=inp["slots"], mask=inp["mask"])
            delta.keep(*x[1:], inp["idx"], inp["n_keep"], slots=inp["slots"])
        return [o, delta.states]
    if kind == "verify":
        idx = torch.empty_like(inp["tokens"])
        n_keep, nxt = torch.empty(2, case["B"], dtype=torch.int32, device=DEV)
        P.pace_verify(inp["tokens"], inp["p"], inp["q"], inp["u"], idx, n_keep, nxt, mask=inp["mask"])
        return [idx, n_keep, nxt]
    pages, table, lens = st["pages"], inp["table"], inp["lens"]
    if kind == "pages":
        B = case["B"]
        if case["samples"] > 1:
            pages.select(table, lens, src=inp["fork"])
        fits = torch.empty(B, dtype=torch.int32, device=DEV)
        pages.take(table, lens, inp["n_new"], fits)
        if case["copy"]:
            st["kv"].copy_pages(pages)
        seen = table.clone()
        pages.select(table, lens, src=inp["back"])
        return [seen, fits, pages.refs, table, lens] + ([st["kv"].pages()] if case["copy"] else [])
    table = table.clone()
    pages.refs.copy_(inp["refs"])
    pages.compact(table)
    st["kv"].copy_pages(pages)
    return [table, pages.refs, st["kv"].pages()]


# ---- plain form -------------------------------------------------------------------------------------------------------------
def _masked(inp, T):
    """Tokens [B, T] that exist, as 0 or 1."""
    if inp["n_new"] is None:
        return None
    return (torch.arange(T, device=DEV) < inp["n_new"][:, None])


def _plain_delta(q, k, v, a, beta, S, anc=None):
    """Chunks of CHUNK tokens from states S [B, H, d, d] (anc: one chunk, a tree's ancestors [B, T, T]); all fp32, [B, T, H, ..].
    Returns o and the states after the last chunk."""
    B, T, H, d = v.shape
    C = min(CHUNK, T) if anc is None else T
    n = -(-T // C)
    pad = n * C - T

    def split(x, fill=0.0):
        x = torch.cat((x, x.new_full((B, pad) + x.shape[2:], fill)), 1) if pad else x
        return x.view((B, n, C) + x.shape[2:]).transpose(2, 3).transpose(1, 2)          # [B, H, n, C, ..]

    g = H // k.shape[2]
    k, q = split(k).repeat_interleave(g, 1), split(q).repeat_interleave(g, 1)
    v, a, beta = split(v), split(a, 1.0), split(beta)
    see = torch.ones(C, C, dtype=torch.bool, device=DEV).tril() if anc is None else anc[:, None, None]
    # R[t, s]: product of the decays of t's ancestors after s; G[t]: of all of them
    log = torch.log(a.double())
    path = (see.double() * log[..., None, :]).sum(-1)
    R = torch.where(see, torch.exp(path[..., :, None] - path[..., None, :]).float(), 0.0)
    G = torch.exp(path).float()[..., None]
    A = (k @ k.transpose(-1, -2)) * R * beta[..., None]
    A = A.masked_fill(torch.eye(C, dtype=torch.bool, device=DEV), 0.0)
    # (I + A)^-1 applied to beta v and beta G k, row by row
    rhs = torch.cat((beta[..., None] * v, beta[..., None] * G * k), -1)
    for t in range(1, C):
        rhs[..., t, :] -= (A[..., t, :t, None] * rhs[..., :t, :]).sum(-2)
    U, W = rhs[..., :d], rhs[..., d:]
    Pq = (q @ k.transpose(-1, -2)) * R
    out = []
    for c in range(n):
        u = U[:, :, c] - W[:, :, c] @ S
        out.append(G[:, :, c] * (q[:, :, c] @ S) + Pq[:, :, c] @ u)
        if anc is None:
            S = G[:, :, c, -1:] * S + (k[:, :, c] * R[:, :, c, -1, :, None]).transpose(-1, -2) @ u
    return torch.stack(out, 2).transpose(1, 2).transpose(2, 3).reshape(B, n * C, H, d)[:, :T], S


def _run_plain_delta(st):
    case, inp = st["case"], st["inp"]
    B, T, dt = case["B"], case["T"], _dt(case)
    q, k, v, a, beta = (inp[n].float() for n in ("q", "k", "v", "a", "beta"))
    at = inp["slots"].long()
    S = inp["states"][at]
    if case["kind"] == "chunk":
        live = _masked(inp, T)
        if live is not None:
            a, beta = torch.where(live[..., None], a, 1.0), beta * live[..., None]
        if inp["lens"] is not None:
            S = S * (inp["lens"] > 0)[:, None, None, None]
        o, S = _plain_delta(q, k, v, a, beta, S)
        if live is not None:
            o = o * live[..., None, None]
        inp["states"][at] = S
        return [o.to(dt), inp["states"]]
    o, _ = _plain_delta(q, k, v, a, beta, S, inp["anc"])
    pick, live = inp["idx"].long(), torch.arange(T, device=DEV) < inp["n_keep"][:, None]
    k, v, a, beta = (torch.gather(x, 1, pick.view((B, T) + (1,) * (x.dim() - 2)).expand(x.shape)) for x in (k, v, a, beta))
    _, S = _plain_delta(k, k, v, torch.where(live[..., None], a, 1.0), beta * live[..., None], S)
    inp["states"][at] = S
    return [o.to(dt), inp["states"]]


def _run_plain_verify(st):
    inp = st["inp"]
    tok, u, par = inp["tokens"].long(), inp["u"].double(), inp["parents"]
    B, N = tok.shape
    row = torch.arange(B, device=DEV)
    cur, Z = torch.zeros(B, dtype=torch.long, device=DEV), torch.ones(B, dtype=torch.float64, device=DEV)
    left = inp["p"][:, 0].double()                                        # what the children of `cur` so far leave
    kept = torch.zeros(B, N, dtype=torch.bool, device=DEV)
    kept[:, 0] = True
    for i in range(1, N):
        y, asked = tok[:, i], par[:, i] == cur
        draft = inp["q"][row, cur].double() if inp["q"] is not None else torch.zeros_like(left).scatter_(1, y[:, None], 1.0)
        ok = asked & (u[:, i] * draft[row, y] * Z < left[row, y])
        if inp["q"] is None:                                              # (the draft named y and nothing else)
            less, rest = left.scatter(1, y[:, None], 0.0), (Z - left[row, y]).clamp(min=0.0)
        else:
            less = (left - draft * Z[:, None]).clamp(min=0.0)
            rest = less.sum(1)
        no = asked & ~ok
        left = torch.where(ok[:, None], inp["p"][:, i].double(), torch.where(no[:, None], less, left))
        Z = torch.where(ok, torch.ones_like(Z), torch.where(no, rest, Z))
        cur = torch.where(ok, torch.full_like(cur, i), cur)
        kept[:, i] = ok
    left = torch.where(left.sum(1, keepdim=True) > 0, left, inp["p"][row, cur].double())
    cum = left.cumsum(1)
    total = left.sum(1)
    over = cum > (u[:, 0] * total)[:, None]
    V = torch.arange(left.shape[1], device=DEV)
    first = torch.where(over & (left > 0), V, left.shape[1]).amin(1)
    last = torch.where(left > 0, V, -1).amax(1)
    nxt = torch.where(first < left.shape[1], first, last)
    order = torch.where(kept, torch.arange(N, device=DEV), N).sort(1).values
    n_keep = kept.sum(1)
    idx = torch.where(order == N, torch.gather(order, 1, n_keep[:, None] - 1), order)
    return [idx.int(), n_keep.int(), nxt.int()]


def _plain_select(table, lens, refs, src, page):
    B, C = table.shape
    n = torch.where(src >= 0, lens[src.clamp(min=0).long()], 0)
    new = torch.where(torch.arange(C, device=DEV) < ((n + page - 1) // page)[:, None], table[src.clamp(min=0).long()], -1)
    for t, d in ((new, 1), (table, -1)):
        held = t >= 0
        refs.index_add_(0, t.clamp(min=0).flatten().long(), held.flatten().int() * d)
    table.copy_(new)
    lens.copy_(n)


def _plain_take(table, lens, refs, n_new, page):
    """Pages for the slots lens .. lens + n_new - 1 of each row: a copy of a shared page that they begin in, and new ones. The
    lowest free pages go out in row order; a row that the pool cannot serve gets none."""
    B, C = table.shape
    col = torch.arange(C, device=DEV)
    c0, end = lens // page, (lens + n_new + page - 1) // page
    inside = (lens % page > 0) & (n_new > 0)
    cell = torch.gather(table, 1, c0[:, None].long().clamp(max=C - 1))[:, 0]
    same = (cell[:, None] == cell[None]) & inside[None]
    writers = same.sum(1)
    lowest = (same.int().cumsum(1) == 1).int().argmax(1) == torch.arange(B, device=DEV)
    shared = refs[cell.clamp(min=0).long()]
    copy = inside & (shared > 1) & ~((writers == shared) & lowest)
    want = (table < 0) & (col >= ((lens + page - 1) // page)[:, None]) & (col < end[:, None]) & (n_new > 0)[:, None]
    want |= copy[:, None] & (col == c0[:, None])
    need = want.sum(1)
    free = torch.nonzero(refs == 0)[:, 0].int()
    fits = (need.cumsum(0) <= free.numel()) | (need == 0)
    want &= fits[:, None]
    copy &= fits
    rank = (want.flatten().cumsum(0) - 1).view(B, C)
    got = torch.cat((free, free.new_zeros(1)))[rank.clamp(0, free.numel())]
    moves = torch.stack((cell, torch.gather(got, 1, c0[:, None].long().clamp(max=C - 1))[:, 0]))[:, copy].long()
    refs[got[want].long()] = 1
    refs.index_add_(0, moves[0], torch.full_like(moves[0], -1, dtype=torch.int32))
    table.copy_(torch.where(want, got, table))
    return fits.int(), moves


def _run_plain_pages(st):
    case, inp = st["case"], st["inp"]
    page, refs, lens = case["page"], inp["refs"], inp["lens"]
    if case["kind"] == "compact":
        table, refs = inp["table"].clone(), refs.clone()
        used = refs > 0
        n = int(used.sum())
        src, dst = torch.nonzero(used[n:])[:, 0] + n, torch.nonzero(~used[:n])[:, 0]
        to = torch.arange(refs.numel(), device=DEV)
        to[src] = dst
        refs[dst] = refs[src]
        refs[src] = 0
        table = torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table)
        inp["pool"][dst] = inp["pool"][src]
        return [table, refs, inp["pool"]]
    table = inp["table"]
    if case["samples"] > 1:
        _plain_select(table, lens, refs, inp["fork"], page)
    fits, moves = _plain_take(table, lens, refs, inp["n_new"], page)
    if case["copy"]:
        inp["pool"][moves[1]] = inp["pool"][moves[0]]
    seen = table.clone()
    _plain_select(table, lens, refs, inp["back"], page)
    return [seen, fits, refs, table, lens] + ([inp["pool"]] if case["copy"] else [])


def _run_plain(st):
    kind = st["case"]["kind"]
    if kind in ("chunk", "draft"):
        return _run_plain_delta(st)
    return _run_plain_verify(st) if kind == "verify" else _run_plain_pages(st)


# ---- the definition in 64 bits ------------------------------------------------------------------------------------------------
def _x_rule(S, q, k, v, a, beta):
    """One token: S [B, H, d, d], the others [B, H, ..]; returns the new state and (with q) the output."""
    S = a[..., None, None] * S
    u = beta[..., None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    return S, None if q is None else (S * q[..., None]).sum(-2)


def exact(case, seed):
    if case["kind"] not in ("chunk", "draft"):
        return None                                      # whole numbers
    B, T, H = case["B"], case["T"], case["H"]
    size = B * H * case["d"] ** 2
    if T * (size * 8 * 6 / 5e12 + 1.5e-4) > 18:
        return None
    inp = _inputs(case, seed)
    g = H // case["Hk"]
    q, k = (inp[n].double().repeat_interleave(g, 2) for n in ("q", "k"))
    v, a, beta = (inp[n].double() for n in ("v", "a", "beta"))
    states = inp["states"].double()
    at = inp["slots"].long()
    S = states[at]
    o = torch.zeros_like(v)
    if case["kind"] == "chunk":
        if inp["lens"] is not None:
            S = torch.where((inp["lens"] > 0)[:, None, None, None], S, 0.0)
        for t in range(T):
            on = torch.ones(B, dtype=torch.bool, device=DEV) if inp["n_new"] is None else inp["n_new"] > t
            new, y = _x_rule(S, q[:, t], k[:, t], v[:, t], a[:, t], beta[:, t])
            S = torch.where(on[:, None, None, None], new, S)
            o[:, t] = torch.where(on[:, None, None], y, 0.0)
        states[at] = S
        return [o, states]
    row = torch.arange(B, device=DEV)
    for t in range(T):                                   # along the path to each node, from the start
        X = S
        for s in range(t + 1):
            new, y = _x_rule(X, q[:, s], k[:, s], v[:, s], a[:, s], beta[:, s])
            X = torch.where(inp["anc"][:, t, s, None, None, None], new, X)
        o[:, t] = y
    for i in range(int(inp["n_keep"].max())):
        s = inp["idx"][:, i].long()
        new, _ = _x_rule(S, None, k[row, s], v[row, s], a[row, s], beta[row, s])
        S = torch.where((inp["n_keep"] > i)[:, None, None, None], new, S)
    states[at] = S
    return [o, states]
