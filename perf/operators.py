"""Measured cases of the attention-layer operators: rotary positions, the quantized paged KV cache (write with rotation, read
back, keep an accepted path) and attention over it (single tokens, trees of drafted tokens, prompt chunks).

`own` False computes every pass in plain torch operations in 32 bits; `own` True makes the calls a user of
bit_gated_delta_gb300 makes. Both read the same seeded inputs.

Cache format (both sides): groups of 64 elements along the head. 8 bits: s = bf16(max|x| / 127), c = clamp(rint(x * (1/s)), -127,
127), value s*c. 4 bits: lo = min(0, x), hi = max(0, x), s = bf16((hi - lo) / 15), z = clamp(rint(-lo * (1/s)), 0, 15),
u = clamp(rint(x * (1/s)) + z, 0, 15), value s*(u - z). Each operation rounds once to fp32; a zero or subnormal s makes the
group zero.
"""
import math

import torch

own = False

GROUP = 64
DEV = "cuda"
ROPE_BASE = 10000.0
FILL = 2048                      # tokens a sequence of one fill chunk


def _dt(case):
    return torch.float32 if case["io"] == "f32" else torch.bfloat16


def listed():
    return [
        # queries of one decode step of a 48-head layer with interleaved pairs on half the head, long-context scaling
        dict(name="rope_decode", kind="rope", N=16, H=48, d=128, rot=64, layout="interleaved", scaling="parts", io="f32",
             max_pos=32768),
        # queries of a prompt chunk: 64 sequences x 256 tokens, 32 heads, whole head rotated in halves
        dict(name="rope_prompt", kind="rope", N=16384, H=32, d=128, rot=128, layout="half", scaling="none", io="bf16",
             max_pos=4096),
        # one decode token of 64 sequences written at 4 bits with rotation, and read back
        dict(name="append_decode", kind="append", B=64, T=1, Hq=32, Hkv=8, d=128, bits=4, io="bf16", lo=300, hi=512, page=64,
             rot=128, layout="half", scaling="none"),
        # a 256-token prompt chunk of 16 long sequences at 8 bits, a quarter of the head rotated, read back
        dict(name="append_prompt", kind="append", B=16, T=256, Hq=48, Hkv=8, d=128, bits=8, io="bf16", lo=1000, hi=4000,
             page=128, rot=32, layout="half", scaling="linear"),
        # a long 4-bit cache read back whole (checkpoint, recomputation)
        dict(name="read_long", kind="read", B=4, Hkv=8, d=128, bits=4, io="bf16", lo=20000, hi=32768, page=64),
        # one user, short context, one token: the latency of a small call
        dict(name="attend_one", kind="attend", B=1, T=1, Hq=16, Hkv=4, d=64, bits=8, io="f32", lo=300, hi=300, page=32,
             tree=False),
        # a serving batch of 64 ragged contexts, one token each, 4-bit cache
        dict(name="attend_batch", kind="attend", B=64, T=1, Hq=32, Hkv=8, d=128, bits=4, io="bf16", lo=512, hi=4096, page=64,
             tree=False),
        # the long-context layer: 48 heads, 16 sequences of about 32k tokens, 8-bit cache
        dict(name="attend_long", kind="attend", B=16, T=1, Hq=48, Hkv=8, d=128, bits=8, io="bf16", lo=30001, hi=32767,
             page=128, tree=False),
        # 25 drafted tokens a sequence as a tree over 4k contexts, 4-bit cache
        dict(name="attend_tree", kind="attend", B=16, T=25, Hq=32, Hkv=8, d=128, bits=4, io="bf16", lo=2049, hi=4096, page=64,
             tree=True),
        # a 256-token prompt chunk attending causally to itself and about 8k cached tokens
        dict(name="attend_prompt", kind="attend", B=4, T=256, Hq=32, Hkv=8, d=128, bits=4, io="bf16", lo=6000, hi=8000,
             page=64, tree=False),
        # one speculative step of a small head: write 16 drafts, attend as a tree, keep the accepted path, read it
        dict(name="step_small", kind="step", B=8, T=16, Hq=16, Hkv=2, d=64, bits=8, io="bf16", lo=500, hi=1500, page=32,
             tree=True, rot=64, layout="interleaved", scaling="ntk"),
        # the same for wide heads and a larger batch, 4-bit cache
        dict(name="step_wide", kind="step", B=32, T=7, Hq=16, Hkv=2, d=256, bits=4, io="bf16", lo=1000, hi=6000, page=64,
             tree=True, rot=64, layout="half", scaling="parts"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.0e15


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        kind = rng.choice(["rope", "append", "read", "attend", "attend", "attend", "step"])
        d = rng.choice([64, 128, 128, 256])
        rot = rng.choice([d, d // 2, 32, 64])
        pos = dict(rot=rot, layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "parts"]))
        io = rng.choice(["bf16", "bf16", "bf16", "f32"])
        if kind == "rope":
            case = dict(kind=kind, N=_log_int(rng, 1, 16384), H=rng.randint(1, 48), d=d, io=io,
                        max_pos=rng.choice([4096, 32768]), **pos)
        else:
            hkv = rng.choice([1, 2, 3, 4, 5, 8])
            base = dict(kind=kind, Hkv=hkv, d=d, bits=rng.choice([4, 8]), io=io, page=rng.choice([32, 64, 128]))
            grp = rng.choice([1, 2, 3, 4, 6, 7, 8])
            hi = _log_int(rng, 100, 32768)
            lo = max(1, int(hi * rng.uniform(0.3, 1.0)))
            if kind == "read":
                case = dict(base, B=_log_int(rng, 1, 64), lo=lo, hi=hi)
            elif kind == "append":
                case = dict(base, B=_log_int(rng, 1, 64), T=_log_int(rng, 1, 256), Hq=hkv * grp, lo=min(lo, 4000),
                            hi=min(hi, 4000), **pos)
            elif kind == "attend":
                tree = rng.random() < 0.4
                case = dict(base, B=_log_int(rng, 1, 64), T=1 if rng.random() < 0.4 else _log_int(rng, 2, 64 if tree else 256),
                            Hq=hkv * grp, lo=lo, hi=hi, tree=tree)
            else:
                case = dict(base, B=_log_int(rng, 1, 32), T=_log_int(rng, 2, 64), Hq=hkv * grp, lo=min(lo, 8000),
                            hi=min(hi, 8000), tree=True, **pos)
            slots = case["B"] * case["hi"] * hkv * d
            if slots > 16 * 32768 * 8 * 128 or case["B"] * case.get("T", 1) * case.get("Hq", 1) * case["hi"] > 2.7e8:
                continue
        if case["H" if kind == "rope" else "Hkv"] * d != 3072 and case.get("Hq", 0) * d != 3072 and _cost(case) <= top:
            return case


def _lens(case):
    """Ragged context lengths of the case, the same for every seed."""
    lo, hi = case["lo"], case["hi"]
    return [lo + int((hi - lo) * ((b * 0.6180339887498949 + 0.5) % 1.0)) for b in range(case["B"])]


def _row_bytes(case):
    """Bytes one cached (token, head) takes: codes, bf16 scales and (4 bits) zero points of k and v."""
    ng = case["d"] // GROUP
    return 2 * (case["d"] * case["bits"] // 8 + 2 * ng + (ng if case["bits"] == 4 else 0))


def work(case):
    es = 4 if case["io"] == "f32" else 2
    kind = case["kind"]
    if kind == "rope":
        n, h, d, rot = case["N"], case["H"], case["d"], case["rot"]
        return {"bytes": 2 * n * h * d * es + n * (4 + rot * 4), "flops": 3 * n * h * rot}
    b, hkv, d = case["B"], case["Hkv"], case["d"]
    lens, row = _lens(case), _row_bytes(case)
    if kind == "read":
        n = sum(lens) * hkv
        return {"bytes": n * (row + 2 * d * es), "flops": 4 * n * d}
    t, hq = case["T"], case["Hq"]
    write = b * t * (2 * hq * d * es + hkv * (2 * d * es + row) + case.get("rot", 0) * 4)
    if kind == "append":
        return {"bytes": write + b * t * hkv * (row + 2 * d * es), "flops": b * t * (3 * (hq + hkv) * case["rot"] + 8 * hkv * d)}
    seen = (lambda n: t * n + t) if case["tree"] else (lambda n: t * n + t * (t + 1) // 2)
    att = {"bytes": sum(n + t for n in lens) * hkv * row + 2 * b * t * hq * d * es,
           "flops": 4 * hq * d * sum(seen(n) for n in lens)}
    if kind == "step":
        att["bytes"] += write + b * (t + 1) // 2 * hkv * (2 * row + 2 * d * es)
    return att


# ---- inputs ---------------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(gen, shape, dtype, amp=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * amp).to(dtype)


def _inputs(case, seed):
    """The seeded inputs both forms and `exact` start from."""
    g = _gen(seed)
    dt = _dt(case)
    if case["kind"] == "rope":
        return dict(x=_randn(g, (case["N"], case["H"], case["d"]), dt),
                    pos=torch.randint(0, case["max_pos"], (case["N"],), generator=g, device=DEV, dtype=torch.int32))
    B, Hkv, d, P = case["B"], case["Hkv"], case["d"], case["page"]
    T = case.get("T", 0)
    lens = _lens(case)
    mp = (max(lens) + T + P - 1) // P
    need = [(n + T + P - 1) // P for n in lens]
    order = torch.randperm(sum(need), generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(B, mp, dtype=torch.int32, device=DEV)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    inp = dict(lens=torch.tensor(lens, dtype=torch.int32, device=DEV), table=table, n_pages=sum(need))
    # a few key channels are larger for every token, as trained keys have them
    amp = torch.ones(Hkv, d, device=DEV)
    amp.scatter_(1, torch.randint(0, d, (Hkv, 4), generator=g, device=DEV), 4.0)
    inp["amp"] = amp
    inp["fill_seed"] = int(torch.randint(0, 2 ** 31 - 1, (1,), generator=g, device=DEV).item())
    if T:
        Hq = case["Hq"]
        inp["q"] = _randn(g, (B, T, Hq, d), dt, 1.5)
        inp["k"] = (torch.randn((B, T, Hkv, d), generator=g, device=DEV) * amp).to(dt)
        inp["v"] = _randn(g, (B, T, Hkv, d), dt)
        if case.get("tree"):
            _tree(case, g, inp)
        else:
            inp["mask"] = None
            inp["pos"] = (inp["lens"][:, None] + torch.arange(T, device=DEV, dtype=torch.int32)).contiguous()
    return inp


def _tree(case, g, inp):
    """A tree of T drafted tokens a sequence: each hangs from the context or from an earlier draft. Ancestor bits (itself
    among them) as 32-bit words, positions by depth, and the path to one accepted draft."""
    B, T = case["B"], case["T"]
    W = (T + 31) // 32
    u = torch.rand(B, T, generator=g, device=DEV).cpu().tolist()
    pick = torch.randint(0, T, (B,), generator=g, device=DEV).cpu().tolist()
    words, depth, idx, nk = [], [], [], []
    K = (T + 1) // 2
    for b in range(B):
        anc, dep, par = [], [], []
        for t in range(T):
            p = max(-1, t - 1 - int(u[b][t] * 4)) if t else -1
            par.append(p)
            anc.append((anc[p] if p >= 0 else 0) | (1 << t))
            dep.append(dep[p] + 1 if p >= 0 else 0)
        words.append([[(a >> (32 * w)) & 0xFFFFFFFF for w in range(W)] for a in anc])
        depth.append(dep)
        path, t = [], pick[b]
        while t >= 0:
            path.append(t)
            t = par[t]
        path = path[::-1][:K]
        nk.append(len(path))
        idx.append(path + [0] * (K - len(path)))
    m = torch.tensor(words, dtype=torch.int64)
    m = torch.where(m >= 2 ** 31, m - 2 ** 32, m).to(torch.int32)
    inp["mask"] = m.to(DEV)
    inp["pos"] = (inp["lens"].cpu()[:, None] + torch.tensor(depth, dtype=torch.int32)).to(DEV).contiguous()
    inp["idx"] = torch.tensor(idx, dtype=torch.int32, device=DEV)
    inp["n_keep"] = torch.tensor(nk, dtype=torch.int32, device=DEV)


def _fill_chunks(case, inp):
    """(first token, counts, k, v) of the cached context, chunk by chunk."""
    g = _gen(inp["fill_seed"])
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    dt, top = _dt(case), max(_lens(case))
    for c0 in range(0, top, FILL):
        n = min(FILL, top - c0)
        k = (torch.randn((B, n, Hkv, d), generator=g, device=DEV) * inp["amp"]).to(dt)
        v = _randn(g, (B, n, Hkv, d), dt)
        yield c0, (inp["lens"] - c0).clamp(0, n).to(torch.int32), k, v


def _max_pos(case):
    return max(_lens(case)) + case["T"] + 1 if "lo" in case else case["max_pos"]


def _scaling(case):
    """Arguments of the long-context scaling: contexts four times as long as trained."""
    return {"none": dict(), "linear": dict(factor=4.0), "ntk": dict(factor=4.0),
            "parts": dict(factor=4.0, orig_pos=4096)}[case["scaling"]]


# ---- plain form -------------------------------------------------------------------------------------------------------------
def _thetas(case):
    """Angle per position of each pair (64 bits) and the factor on cos and sin."""
    rot, kw = case["rot"], _scaling(case)
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    theta, m = ROPE_BASE ** (-i / rot), 1.0
    if case["scaling"] == "linear":
        theta = theta / kw["factor"]
    elif case["scaling"] == "ntk":
        theta = (ROPE_BASE * kw["factor"] ** (rot / (rot - 2))) ** (-i / rot)
    elif case["scaling"] == "parts":
        turns = kw["orig_pos"] * theta / (2 * math.pi)
        ramp = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        theta = theta * (ramp + (1 - ramp) / kw["factor"])
        m = 0.1 * math.log(kw["factor"]) + 1.0
    return theta, m


def _plain_table(case):
    theta, m = _thetas(case)
    ang = torch.arange(_max_pos(case), dtype=torch.float64, device=DEV)[:, None] * theta.to(DEV)
    return (torch.cos(ang) * m).float(), (torch.sin(ang) * m).float()


def _plain_rotate(x, pos, table, rot, layout):
    """x [..., H, d] in fp32, pos [...]."""
    c, s = table[0][pos.long()].unsqueeze(-2), table[1][pos.long()].unsqueeze(-2)
    h = rot // 2
    if layout == "half":
        a, b = x[..., :h], x[..., h:rot]
        return torch.cat((a * c - b * s, b * c + a * s, x[..., rot:]), -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_quant(x, bits):
    """x [..., d] fp32 -> codes u8, scale fp32 (bf16 values), zero point fp32; per group of 64."""
    g = x.unflatten(-1, (-1, GROUP))
    if bits == 8:
        s = (g.abs().amax(-1) / 127.0).bfloat16().float()
        ok = s >= 1.1754943508222875e-38
        r = torch.where(ok, 1.0 / s, torch.zeros_like(s))
        c = torch.round(g * r.unsqueeze(-1)).clamp(-127, 127)
        z = torch.full_like(s, 128.0)
    else:
        lo, hi = g.amin(-1).clamp(max=0.0), g.amax(-1).clamp(min=0.0)
        s = ((hi - lo) / 15.0).bfloat16().float()
        ok = s >= 1.1754943508222875e-38
        r = torch.where(ok, 1.0 / s, torch.zeros_like(s))
        z = torch.round(-lo * r).clamp(0, 15)
        c = (torch.round(g * r.unsqueeze(-1)) + z.unsqueeze(-1)).clamp(0, 15) - z.unsqueeze(-1)
    s = torch.where(ok, s, torch.zeros_like(s))
    return (c + z.unsqueeze(-1)).to(torch.uint8).flatten(-2), s, z


class _PlainCache:
    """Paged pool, one code a byte."""

    def __init__(self, case, n_pages):
        P, Hkv, d = case["page"], case["Hkv"], case["d"]
        self.P, self.bits = P, case["bits"]
        rows, ng = n_pages * P, d // GROUP
        self.codes = [torch.zeros(rows, Hkv, d, dtype=torch.uint8, device=DEV) for _ in range(2)]
        self.s = [torch.zeros(rows, Hkv, ng, device=DEV) for _ in range(2)]
        self.z = [torch.zeros(rows, Hkv, ng, device=DEV) for _ in range(2)]

    def rows(self, table, slots):
        return torch.gather(table, 1, slots // self.P).long() * self.P + slots % self.P

    def write(self, table, slots, keep, k, v):
        at = self.rows(table, slots.clamp(max=table.shape[1] * self.P - 1))[keep]
        for i, x in enumerate((k, v)):
            c, s, z = _plain_quant(x.float(), self.bits)
            self.codes[i][at], self.s[i][at], self.z[i][at] = c[keep], s[keep], z[keep]

    def values(self, i, at):
        c = self.codes[i][at].float().unflatten(-1, (-1, GROUP))
        return ((c - self.z[i][at].unsqueeze(-1)) * self.s[i][at].unsqueeze(-1)).flatten(-2)

    def read(self, table, first, n, end, dt):
        slots = first.long()[:, None] + torch.arange(n, device=DEV)
        live = slots < end.long()[:, None]
        at = self.rows(table, torch.where(live, slots, torch.zeros_like(slots)))
        return [torch.where(live[..., None, None], self.values(i, at), 0.0).to(dt) for i in range(2)]

    def move(self, table, lens, idx, n_keep):
        j = torch.arange(idx.shape[1], device=DEV)
        live = j < n_keep[:, None]
        src = self.rows(table, lens.long()[:, None] + idx)[live]
        dst = self.rows(table, lens.long()[:, None] + j)[live]
        for arr in (self.codes, self.s, self.z):
            for i in range(2):
                arr[i][dst] = arr[i][src]


def _plain_attend(cache, case, q, table, lens, mask, dt):
    B, T, Hq, d = q.shape
    Hkv = case["Hkv"]
    L = max(_lens(case)) + T
    slots = torch.arange(L, device=DEV)
    at = cache.rows(table, slots.expand(B, L).clamp(max=table.shape[1] * cache.P - 1))
    k = cache.values(0, at).permute(0, 2, 3, 1)                             # [B, Hkv, d, L]
    v = cache.values(1, at).permute(0, 2, 1, 3)
    qg = q.float().view(B, T, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
    s = torch.matmul(qg, k) / math.sqrt(d)
    j = slots[None, :] - lens.long()[:, None]                              # draft index of each slot
    jt = j.clamp(0, T - 1)
    if mask is None:
        draft = jt[:, None, :] <= torch.arange(T, device=DEV)[None, :, None]
    else:
        w = torch.gather(mask, 2, (jt // 32)[:, None, :].expand(B, T, L))
        draft = ((w >> (jt % 32)[:, None, :]) & 1) != 0
    see = (j < 0)[:, None, :] | ((j < T)[:, None, :] & draft)                # [B, T, L]
    see = see[:, None, :, None, :].expand(B, 1, T, Hq // Hkv, L).reshape(B, 1, -1, L)
    s = s.masked_fill(~see, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.view(B, Hkv, T, -1, d).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, d).to(dt)


# ---- the measured interface ---------------------------------------------------------------------------------------------------
def prepare(case, seed):
    st = dict(case=case, inp=_inputs(case, seed))
    inp, kind = st["inp"], case["kind"]
    if own:
        import bit_gated_delta_gb300 as P
        if "rot" in case:
            st["rope"] = P.PaceRope(case["rot"], _max_pos(case), base=ROPE_BASE, scaling=case["scaling"],
                                    layout=case["layout"], **_scaling(case))
        if kind != "rope":
            cfg = P.make_kv_config(q_heads=case.get("Hq", case["Hkv"]), kv_heads=case["Hkv"], d=case["d"], bits=case["bits"],
                                   page_tokens=case["page"], n_pages=inp["n_pages"], max_batch=case["B"], max_new=FILL,
                                   io_dtype=P.PACE_IO_F32 if case["io"] == "f32" else P.PACE_IO_BF16)
            st["kv"] = kv = P.PaceKV(cfg)
            for c0, n, k, v in _fill_chunks(case, inp):
                kv.append(None, k, v, torch.full_like(n, c0), inp["table"], n_new=n)
            if kind == "attend":             # the new tokens are in the cache when attention is called
                kv.append(None, inp["k"], inp["v"], inp["lens"], inp["table"])
    else:
        if "rot" in case:
            st["rope"] = _plain_table(case)
        if kind != "rope":
            st["kv"] = kv = _PlainCache(case, inp["n_pages"])
            for c0, n, k, v in _fill_chunks(case, inp):
                i = torch.arange(k.shape[1], device=DEV)
                kv.write(inp["table"], (c0 + i).expand(case["B"], -1), i < n[:, None], k, v)
            if kind == "attend":
                slots = inp["lens"].long()[:, None] + torch.arange(case["T"], device=DEV)
                kv.write(inp["table"], slots, torch.ones_like(slots, dtype=torch.bool), inp["k"], inp["v"])
    return st


def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import bit_gated_delta_gb300 as P
    case, inp, kind = st["case"], st["inp"], st["case"]["kind"]
    if kind == "rope":
        out = torch.empty_like(inp["x"])
        P.pace_rope_apply(st["rope"], inp["x"], inp["pos"], out)
        return out
    kv, lens, table, dt = st["kv"], inp["lens"], inp["table"], _dt(case)
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    if kind == "read":
        n = max(_lens(case))
        k, v = (torch.empty(B, n, Hkv, d, dtype=dt, device=DEV) for _ in range(2))
        kv.read(k, v, table, end=lens)
        return [k, v]
    q = inp["q"]
    T = case["T"]
    if kind in ("append", "step"):
        q = torch.empty_like(q)
        kv.append(inp["q"], inp["k"], inp["v"], lens, table, rope=st["rope"], positions=inp["pos"], q_out=q)
    if kind == "append":
        k, v = (torch.empty(B, T, Hkv, d, dtype=dt, device=DEV) for _ in range(2))
        kv.read(k, v, table, first=lens)
        return [q, k, v]
    o = torch.empty_like(q)
    kv.attend(q, o, lens, table, mask=inp["mask"])
    if kind == "attend":
        return o
    kv.keep(lens, table, inp["idx"], inp["n_keep"])
    K = inp["idx"].shape[1]
    k, v = (torch.empty(B, K, Hkv, d, dtype=dt, device=DEV) for _ in range(2))
    kv.read(k, v, table, first=lens, end=lens + inp["n_keep"])
    return [o, k, v]


def _run_plain(st):
    case, inp, kind = st["case"], st["inp"], st["case"]["kind"]
    dt = _dt(case)
    if kind == "rope":
        return _plain_rotate(inp["x"].float(), inp["pos"], st["rope"], case["rot"], case["layout"]).to(dt)
    kv, lens, table = st["kv"], inp["lens"], inp["table"]
    if kind == "read":
        return kv.read(table, torch.zeros_like(lens), max(_lens(case)), lens, dt)
    q, T = inp["q"], case["T"]
    if kind in ("append", "step"):
        q = _plain_rotate(q.float(), inp["pos"], st["rope"], case["rot"], case["layout"]).to(dt)
        k = _plain_rotate(inp["k"].float(), inp["pos"], st["rope"], case["rot"], case["layout"])
        slots = lens.long()[:, None] + torch.arange(T, device=DEV)
        kv.write(table, slots, torch.ones_like(slots, dtype=torch.bool), k, inp["v"])
    if kind == "append":
        return [q] + kv.read(table, lens, T, lens + T, dt)
    o = _plain_attend(kv, case, q, table, lens, inp["mask"], dt)
    if kind == "attend":
        return o
    kv.move(table, lens, inp["idx"], inp["n_keep"])
    return [o] + kv.read(table, lens, inp["idx"].shape[1], lens + inp["n_keep"], dt)


# ---- the definition in 64 bits ------------------------------------------------------------------------------------------------
def _x_rotate(case, x, pos):
    """Complex form: each pair (a, b) times m exp(i pos theta)."""
    theta, m = _thetas(case)
    rot = case["rot"]
    ang = pos.double()[..., None, None] * theta.to(DEV)
    w = torch.polar(torch.full_like(ang, m), ang)
    xr = x[..., :rot]
    pairs = xr.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["layout"] == "half" else xr.unflatten(-1, (rot // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
    z = z.transpose(-1, -2).flatten(-2) if case["layout"] == "half" else z.flatten(-2)
    return torch.cat((z, x[..., rot:]), -1)


def _x_held(x, bits):
    """The values the cache holds for x (64 bits in): the format's fp32 roundings, everything else in 64 bits."""
    f32 = lambda y: y.float().double()
    g = f32(x).unflatten(-1, (-1, GROUP))
    top = g.amax(-1, keepdim=True)
    bot = g.amin(-1, keepdim=True)
    if bits == 8:
        s = (torch.maximum(top, -bot) / 127).float().bfloat16().double()
        lo, hi, z = -127, 127, torch.zeros_like(s)
    else:
        top, bot = top.clamp(min=0), bot.clamp(max=0)
        s = (f32(top - bot) / 15).float().bfloat16().double()
        lo, hi = 0, 15
    dead = s < 2.0 ** -126
    inv = f32(1.0 / torch.where(dead, torch.ones_like(s), s))
    if bits == 4:
        z = torch.round(f32(-bot * inv)).clamp(0, 15)
    u = (torch.round(f32(g * inv)) + z).clamp(lo, hi)
    return torch.where(dead, torch.zeros_like(g), (u - z) * s).flatten(-2)


def exact(case, seed):
    inp = _inputs(case, seed)
    kind = case["kind"]
    if kind == "rope":
        return _x_rotate(case, inp["x"].double(), inp["pos"])
    lens, B, Hkv, d = _lens(case), case["B"], case["Hkv"], case["d"]
    T = case.get("T", 0)
    k_new = v_new = q = None
    if T:
        q, k_new, v_new = inp["q"].double(), inp["k"].double(), inp["v"].double()
        if kind != "attend":
            q, k_new = _x_rotate(case, q, inp["pos"]), _x_rotate(case, k_new, inp["pos"])
        k_new, v_new = _x_held(k_new, case["bits"]), _x_held(v_new, case["bits"])
    if kind == "append":
        return [q, k_new, v_new]
    L = max(lens)
    k = torch.zeros(B, L, Hkv, d, dtype=torch.float64, device=DEV)
    v = torch.zeros_like(k)
    for c0, n, kc, vc in _fill_chunks(case, inp):
        live = (torch.arange(kc.shape[1], device=DEV) < n[:, None])[..., None, None]
        k[:, c0:c0 + kc.shape[1]] = torch.where(live, _x_held(kc.double(), case["bits"]), 0.0)
        v[:, c0:c0 + kc.shape[1]] = torch.where(live, _x_held(vc.double(), case["bits"]), 0.0)
    if kind == "read":
        return [k, v]
    if kind == "step":
        q = q.to(_dt(case)).double()         # the step's queries are held in the I/O type between the two calls
    Hq = case["Hq"]
    out = torch.empty(B, T, Hq, d, dtype=torch.float64, device=DEV)
    see = torch.ones(T, T, dtype=torch.bool, device=DEV).tril()
    for b in range(B):
        if inp["mask"] is not None:
            bits = torch.arange(T, device=DEV)
            see = (inp["mask"][b].long()[:, bits // 32] >> (bits % 32)) & 1 != 0
        kb, vb = torch.cat((k[b, :lens[b]], k_new[b])), torch.cat((v[b, :lens[b]], v_new[b]))
        allow = torch.cat((torch.ones(T, lens[b], dtype=torch.bool, device=DEV), see), 1)
        for h in range(Hq):
            kh = h // (Hq // Hkv)
            a = (q[b, :, h] @ kb[:, kh].T) * d ** -0.5
            out[b, :, h] = torch.softmax(a.masked_fill(~allow, -math.inf), -1) @ vb[:, kh]
    if kind == "attend":
        return out
    K = inp["idx"].shape[1]
    live = (torch.arange(K, device=DEV) < inp["n_keep"][:, None])[..., None, None]
    pick = inp["idx"].long()[..., None, None].expand(B, K, Hkv, d)
    return [out] + [torch.where(live, torch.gather(x, 1, pick), 0.0) for x in (k_new, v_new)]
