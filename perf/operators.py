"""Measured cases of the cache operators: rotary positions with the append, decode attention over
shared prefixes (with the weights accumulated per cached token), and eviction by those weights.

``run`` with ``own`` false is the plain form (elementary torch operations in 32 bits); with ``own``
true it makes the calls a user makes.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

BLOCK = 16
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence at a far position: latency
        dict(name="rotary_one", op="rotary", T=1, Hq=32, Hkv=4, d=128, dtype="bf16", rot=128,
             layout="half", scaling="linear", far=1),
        # a decode step of a full batch, part of the head, interleaved, q/k/v slices of one projection
        dict(name="rotary_step256", op="rotary", T=256, Hq=32, Hkv=8, d=128, dtype="bf16", rot=64,
             layout="interleaved", scaling="bands", far=1),
        # prompts of joining sequences, queries and keys, long-context scaling
        dict(name="rotary_prompt16k", op="rotary", T=16384, Hq=32, Hkv=8, d=128, dtype="bf16", rot=128,
             layout="half", scaling="ramp", far=0),
        # a few short chats under one short system prompt: latency
        dict(name="shared_small", op="shared", B=4, Hq=8, Hkv=2, d=64, dtype="bf16", P=1, plo=500,
             phi=500, olo=1, ohi=64, loose=0, mass=0, seed=1),
        # 64 ragged conversations under one 8k prompt
        dict(name="shared_64", op="shared", B=64, Hq=32, Hkv=8, d=128, dtype="bf16", P=1, plo=8192,
             phi=8192, olo=1, ohi=4096, loose=0, mass=0, seed=2),
        # several tenants, each with its own prompt of an odd length, and rows without one
        dict(name="shared_groups256", op="shared", B=256, Hq=32, Hkv=8, d=128, dtype="bf16", P=5,
             plo=777, phi=4097, olo=0, ohi=1023, loose=1, mass=0, seed=3),
        # many questions on one long document: the products dominate
        dict(name="shared_document", op="shared", B=128, Hq=32, Hkv=4, d=128, dtype="bf16", P=1,
             plo=65531, phi=65531, olo=1, ohi=256, loose=0, mass=0, seed=4),
        # a ragged decode step whose weights feed eviction, no prefix
        dict(name="mass_ragged64", op="shared", B=64, Hq=32, Hkv=8, d=128, dtype="bf16", P=0, plo=0,
             phi=0, olo=1, ohi=4096, loose=0, mass=1, seed=5),
        # prefix and weights together in 32 bits
        dict(name="mass_prefix_f32", op="shared", B=24, Hq=16, Hkv=8, d=64, dtype="f32", P=2, plo=250,
             phi=1000, olo=0, ohi=513, loose=1, mass=1, seed=6),
        # small budgets
        dict(name="evict_small", op="evict", B=3, Hkv=2, d=64, dtype="f32", lo=5, hi=200, keep=64,
             sink=4, recent=16, seed=7),
        # a batch brought back to its budget
        dict(name="evict_64", op="evict", B=64, Hkv=8, d=128, dtype="bf16", lo=1500, hi=2600, keep=1024,
             sink=4, recent=256, seed=8),
        # one long context cut to a quarter
        dict(name="evict_long", op="evict", B=1, Hkv=4, d=128, dtype="bf16", lo=131072, hi=131072,
             keep=32768, sink=16, recent=1024, seed=9),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "shared", "shared", "mass", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "rotary":
        rot = rng.choice([d, d, d // 2, d - 32, 16])
        return dict(op=op, T=_spread(rng, 1, 12000), Hq=Hkv * rng.choice([1, 2, 4]), Hkv=Hkv, d=d,
                    dtype=dtype, rot=rot, layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["plain", "linear", "ntk", "ramp", "bands"]),
                    far=rng.choice([0, 1]))
    if op == "evict":
        hi = _spread(rng, 17, 16384)
        keep = max(1, int(hi * rng.uniform(0.1, 0.9)))
        return dict(op=op, B=_spread(rng, 1, max(1, min(64, 131072 // hi))), Hkv=Hkv, d=d, dtype=dtype,
                    lo=max(1, hi // 2), hi=hi, keep=keep, sink=rng.choice([0, 1, 4]),
                    recent=rng.choice([0, 1, keep // 4, keep // 2]), seed=rng.randrange(1 << 20))
    G = rng.choice([1, 2, 4, 8])
    B = _spread(rng, 1, 200)
    f32 = dtype == "f32"
    ohi = _spread(rng, 1, min(4096, 60000 // B))
    phi = _spread(rng, 1, min(16000, (100000 if f32 else 1000000) // B))
    P = rng.choice([1, 1, 2, 5]) if op == "shared" else rng.choice([0, 0, 1, 3])
    return dict(op="shared", B=B, Hq=Hkv * G, Hkv=Hkv, d=d, dtype=dtype, P=P,
                plo=max(1, phi // 3) if P else 0, phi=phi if P else 0, olo=rng.choice([0, 1]), ohi=ohi,
                loose=rng.choice([0, 1]), mass=1 if op == "mass" else rng.choice([0, 0, 1]),
                seed=rng.randrange(1 << 20))


def _lengths(case):
    """Own length and prefix of every row, and the prefixes' lengths (a function of the case)."""
    rng = random.Random(case["seed"])
    own_lens = [rng.randint(case["olo"], case["ohi"]) for _ in range(case["B"])]
    own_lens[-1] = case["ohi"]
    plens = [rng.randint(case["plo"], case["phi"]) for _ in range(case["P"])]
    lowest = -1 if case["loose"] else 0
    rows = [rng.randint(lowest, case["P"] - 1) if case["P"] else -1 for _ in range(case["B"])]
    return own_lens, plens, rows


def _evict_lengths(case):
    rng = random.Random(case["seed"])
    lens = [rng.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    lens[-1] = case["hi"]
    # budgets differ a little from row to row
    keeps = [max(1, case["keep"] - rng.randint(0, case["keep"] // 8)) for _ in range(case["B"])]
    keeps[-1] = case["keep"]
    return lens, keeps


def work(case):
    e, d = ESIZE[case["dtype"]], case["d"]
    Hkv = case["Hkv"]
    if case["op"] == "rotary":
        rows = case["T"] * (case["Hq"] + 2 * Hkv)
        return {"bytes": 2 * rows * d * e + 12 * case["T"], "flops": 3 * rows * d}
    if case["op"] == "evict":
        lens, keeps = _evict_lengths(case)
        b = 0
        for L, K in zip(lens, keeps):
            if K < L:
                b += Hkv * (4 * L + 2 * 2 * K * d * e + 8 * K + 4 * K)
        return {"bytes": max(b, 1), "flops": 0}
    own_lens, plens, rows = _lengths(case)
    used = sum(plens[p] for p in set(rows) if p >= 0)
    b = 2 * (used + sum(own_lens)) * Hkv * d * e + 2 * case["B"] * case["Hq"] * d * e
    if case["mass"]:
        b += 8 * sum(own_lens) * Hkv
    tokens = sum(own_lens) + sum(plens[p] for p in rows if p >= 0)
    return {"bytes": b, "flops": 4 * d * case["Hq"] * tokens}


# --------------------------------------------------------------------------- inputs
def _gen(seed, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1009 + k)
    return g


def _normal(shape, dtype, seed, k):
    out = torch.empty(shape, dtype=DTYPES[dtype], device="cuda")
    g = _gen(seed, k)
    rows = max(1, (1 << 27) // max(1, out[0].numel()))
    for s in range(0, shape[0], rows):
        part = out[s:s + rows]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return out


def _tables(lens, free, at):
    """Block tables [len(lens), most] (int32, -1 padded) taking blocks of `free` from `at` on."""
    need = [-(-n // BLOCK) for n in lens]
    table = torch.full((len(lens), max([1] + need)), -1, dtype=torch.int32)
    for i, n in enumerate(need):
        table[i, :n] = free[at:at + n]
        at += n
    return table, at


def _pool(lens_lists, seed):
    """Scattered tables of several lists of lengths over a pool of 1.25 times the blocks, of which the
    last block drawn belongs to nobody."""
    blocks = sum(-(-n // BLOCK) for lens in lens_lists for n in lens)
    n = blocks + max(1, blocks // 4)
    g = torch.Generator()
    g.manual_seed(seed)
    free = torch.randperm(n, generator=g).to(torch.int32)
    at, got = 0, []
    for lens in lens_lists:
        t, at = _tables(lens, free, at)
        got.append(t)
    return n, got, int(free[-1])


ROTARY = {
    "plain": dict(factor=1.0, low=1.0, high=32.0, original=0, amplitude=1.0),
    "linear": dict(factor=8.0, low=1.0, high=32.0, original=0, amplitude=1.0),
    "ntk": dict(factor=4.0, low=1.0, high=32.0, original=0, amplitude=1.0),
    "ramp": dict(factor=16.0, low=1.0, high=32.0, original=4096, amplitude=1.2772588722239782),
    "bands": dict(factor=8.0, low=1.0, high=4.0, original=8192, amplitude=1.0),
}
BASE = {"plain": 10000.0, "linear": 10000.0, "ntk": 10000.0, "ramp": 10000.0, "bands": 500000.0}


def prepare(case, seed):
    if case["op"] == "rotary":
        return _prepare_rotary(case, seed)
    if case["op"] == "evict":
        return _prepare_evict(case, seed)
    return _prepare_shared(case, seed)


def _prepare_rotary(case, seed):
    T, Hq, Hkv, d, dt = case["T"], case["Hq"], case["Hkv"], case["d"], case["dtype"]
    qkv = _normal((T, Hq + 2 * Hkv, d), dt, seed, 1)   # one projection's output: q, k, v side by side
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    rng = random.Random(seed)
    if case["far"]:    # every token at its own far position, in a block of its own
        pos = torch.tensor([rng.randrange(1 << 17) for _ in range(T)], dtype=torch.int32)
        n, (tab,), _ = _pool([[BLOCK] * T], seed)
        slots = tab[:, 0].to(torch.int64) * BLOCK + pos.to(torch.int64) % BLOCK
    else:              # prompts, one after another
        pos = torch.arange(T, dtype=torch.int32) % 6000
        n, (tab,), _ = _pool([[T]], seed)
        t = torch.arange(T)
        slots = tab[0].to(torch.int64)[t // BLOCK] * BLOCK + t % BLOCK
    s = dict(case=case, q=q, k=k, v=v, pos=pos.cuda(), slots=slots.cuda(),
             k_cache=_normal((n, Hkv, BLOCK, d), dt, seed, 2),
             v_cache=_normal((n, Hkv, BLOCK, d), dt, seed, 3))
    if own:
        from paged_kv_decode_10_gb300 import binding
        p = ROTARY[case["scaling"]]
        rot = binding.Rotary(d, rot_dim=case["rot"], layout=case["layout"], scaling=case["scaling"],
                             base=BASE[case["scaling"]], factor=p["factor"], low=p["low"],
                             high=p["high"], original_len=p["original"], amplitude=p["amplitude"])
        s["q_out"] = torch.empty((T, Hq, d), dtype=DTYPES[dt], device="cuda")
        s["args"] = binding.make_rotary_args(rot, q, k, v, s["pos"], q_out=s["q_out"],
                                             slot_mapping=s["slots"], k_cache=s["k_cache"],
                                             v_cache=s["v_cache"])
    return s


def _prepare_shared(case, seed):
    B, Hq, Hkv, d, dt = case["B"], case["Hq"], case["Hkv"], case["d"], case["dtype"]
    own_lens, plens, rows = _lengths(case)
    n, (tab, ptab), spare = _pool([own_lens, plens], seed)
    s = dict(case=case, scale=1.0 / math.sqrt(d), spare=spare, plens=plens, rows=rows,
             longest=max(own_lens), q=_normal((B, Hq, d), dt, seed, 1),
             k_cache=_normal((n, Hkv, BLOCK, d), dt, seed, 2),
             v_cache=_normal((n, Hkv, BLOCK, d), dt, seed, 3), tables=tab.cuda(),
             ptables=ptab.cuda(), lens=torch.tensor(own_lens, dtype=torch.int32).cuda())
    if case["mass"]:
        s["mass"] = torch.rand((n, Hkv, BLOCK), generator=_gen(seed, 4), device="cuda")
        # the newest token of every row has no weight yet
        s["mass_lens"] = (s["lens"] - 1).clamp(min=0)
    if case["P"]:
        # rows of each prefix (padded with the batch size), as a server knows them
        lists = [[b for b in range(B) if rows[b] == p] for p in range(case["P"])]
        most = max([1] + [len(x) for x in lists])
        s["members"] = torch.tensor([x + [B] * (most - len(x)) for x in lists]).cuda()
        s["plens_dev"] = torch.tensor(plens, dtype=torch.int32).cuda()
    if own:
        from paged_kv_decode_10_gb300 import binding
        s["out"] = torch.empty((B, Hq, d), dtype=DTYPES[dt], device="cuda")
        kw = {}
        if case["P"]:
            plan = binding.shared_plan(rows, plens, Hq, Hkv, d, binding.dtype_code(s["q"]))
            kw.update(prefix_tables=s["ptables"], prefix_plan=torch.from_numpy(plan).cuda())
        if case["mass"]:
            s["scores"] = binding.alloc_scores(n, Hq, s["q"].device)
            kw.update(mass=s["mass"], scores=s["scores"], mass_lens=s["mass_lens"], decay=0.9375)
        s["args"] = binding.make_shared_args(s["q"], s["k_cache"], s["v_cache"], s["tables"],
                                             s["lens"], s["scale"], s["out"], **kw)
    return s


def _prepare_evict(case, seed):
    B, Hkv, d, dt = case["B"], case["Hkv"], case["d"], case["dtype"]
    lens, keeps = _evict_lengths(case)
    n, (tab,), spare = _pool([lens], seed)
    # accumulated weights are heavy-tailed, and some tokens were never attended to at all
    mass = torch.randn((n, Hkv, BLOCK), generator=_gen(seed, 4), device="cuda").mul_(2.0).exp_()
    mass *= (torch.rand(mass.shape, generator=_gen(seed, 5), device="cuda") > 0.1)
    s = dict(case=case, spare=spare, longest=max(lens), most=max(keeps), tables=tab.cuda(),
             lens=torch.tensor(lens, dtype=torch.int32).cuda(),
             keeps=torch.tensor(keeps, dtype=torch.int32).cuda(), mass=mass,
             k_cache=_normal((n, Hkv, BLOCK, d), dt, seed, 2),
             v_cache=_normal((n, Hkv, BLOCK, d), dt, seed, 3))
    if own:
        from paged_kv_decode_10_gb300 import binding
        s["kept"] = torch.empty((B, Hkv, s["most"]), dtype=torch.int32, device="cuda")
        s["args"] = binding.make_evict_args(s["k_cache"], s["v_cache"], mass, s["tables"], s["lens"],
                                            s["keeps"], s["kept"], sink=case["sink"],
                                            recent=case["recent"])
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        from paged_kv_decode_10_gb300 import binding
        if op == "rotary":
            binding.rotary_append_args(s["args"])
            return s["q_out"], s["k_cache"], s["v_cache"]
        if op == "evict":
            binding.evict_args(s["args"])
            return s["kept"], s["k_cache"], s["v_cache"], s["mass"]
        binding.decode_attn_shared_args(s["args"])
        return (s["out"], s["mass"]) if s["case"]["mass"] else s["out"]
    if op == "rotary":
        return _plain_rotary(s)
    if op == "evict":
        return _plain_evict(s)
    return _plain_shared(s)


def _frequencies(case):
    """Radians per position of every rotated pair, in 64 bits."""
    r, p, base = case["rot"], ROTARY[case["scaling"]], BASE[case["scaling"]]
    F, N = p["factor"], p["original"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    if case["scaling"] == "ntk":
        base = base * F ** (r / (r - 2))
    f = base ** (-2.0 * i / r)
    if case["scaling"] == "linear":
        f = f / F
    elif case["scaling"] == "ramp":
        lo = math.floor(r * math.log(N / (2 * math.pi * p["high"])) / (2 * math.log(base)))
        hi = math.ceil(r * math.log(N / (2 * math.pi * p["low"])) / (2 * math.log(base)))
        lo, hi = max(lo, 0), min(hi, r - 1)
        g = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - g) + f / F * g
    elif case["scaling"] == "bands":
        g = ((N * f / (2 * math.pi) - p["low"]) / (p["high"] - p["low"])).clamp(0, 1)
        f = f * g + f / F * (1 - g)
    return f


def _plain_rotary(s):
    case = s["case"]
    r, half, dt = case["rot"], case["rot"] // 2, DTYPES[case["dtype"]]
    a = ROTARY[case["scaling"]]["amplitude"]
    theta = s["pos"].double()[:, None] * _frequencies(case)
    cos, sin = (a * theta.cos()).float()[:, None], (a * theta.sin()).float()[:, None]

    def turn(x):
        y = x.float()
        x1, x2 = (y[..., :half], y[..., half:r]) if case["layout"] == "half" else (y[..., 0:r:2],
                                                                                  y[..., 1:r:2])
        z1, z2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
        if case["layout"] == "half":
            z = torch.cat([z1, z2], -1)
        else:
            z = torch.stack([z1, z2], -1).flatten(-2)
        return torch.cat([z, y[..., r:]], -1).to(dt)

    blk, row = s["slots"] // BLOCK, s["slots"] % BLOCK
    s["k_cache"][blk, :, row] = turn(s["k"])
    s["v_cache"][blk, :, row] = s["v"]
    return turn(s["q"]), s["k_cache"], s["v_cache"]


def _part(q, k, v, ok):
    """Softmax attention of q [..., M, d] over k, v [..., L, d] where ok [..., 1, L]: the largest
    score, the weights (relative to it), their sum and the weighted values."""
    score = (q @ k.transpose(-1, -2)).masked_fill_(~ok, -math.inf)
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - m.masked_fill(m == -math.inf, 0.0))
    return m, p, p.sum(-1, keepdim=True), p @ v


def _plain_shared(s):
    case = s["case"]
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    G = Hq // Hkv
    q = (s["q"].float() * s["scale"]).view(B, Hkv, G, d)

    def tokens(cache, tables, n):
        t = torch.arange(n, device="cuda")
        blk = tables.long()[:, t // BLOCK]
        blk = torch.where(blk < 0, s["spare"], blk)
        return cache[blk, :, t % BLOCK].float().transpose(1, 2), blk, t   # [rows, Hkv, n, d]

    n = max(s["longest"], 1)
    k, blk, t = tokens(s["k_cache"], s["tables"], n)
    v = tokens(s["v_cache"], s["tables"], n)[0]
    ok = (t < s["lens"][:, None])[:, None, None]
    m, p, l, o = _part(q, k, v, ok)
    o.masked_fill_(l == 0, 0.0)
    M = m
    if case["P"]:
        most = s["members"].shape[1]
        longest = max(s["plens"])
        qp = torch.cat([q, q.new_zeros(1, Hkv, G, d)])[s["members"]]      # [P, most, Hkv, G, d]
        qp = qp.transpose(1, 2).reshape(case["P"], Hkv, most * G, d)
        kp, vp = (tokens(c, s["ptables"], longest)[0] for c in (s["k_cache"], s["v_cache"]))
        okp = (torch.arange(longest, device="cuda") < s["plens_dev"][:, None])[:, None, None]
        mp, _, lp, op = _part(qp, kp, vp, okp)
        # back to rows (padding lands in a row of its own behind the batch)
        at = s["members"].reshape(-1)

        def rows(x, empty):
            x = x.view(case["P"], Hkv, most, G, -1).transpose(1, 2).reshape(-1, Hkv, G, x.shape[-1])
            full = x.new_full((B + 1,) + x.shape[1:], empty)
            full[at] = x
            return full[:B]

        mp, lp, op = rows(mp, -math.inf), rows(lp, 0.0), rows(op, 0.0)
        M = torch.maximum(m, mp)
        zero = M.masked_fill(M == -math.inf, 0.0)
        wo, wp = torch.exp(m - zero), torch.exp(mp - zero)
        o, l = o * wo + op * wp, l * wo + lp * wp
    out = (o / torch.where(l > 0, l, 1.0)).view(B, Hq, d).to(s["q"].dtype)
    if not case["mass"]:
        return out
    # each cached token's weight, summed over the group's heads
    rel = torch.exp(m - M.masked_fill(M == -math.inf, 0.0))
    w = (p * rel / torch.where(l > 0, l, 1.0)).sum(2).transpose(1, 2)     # [B, n, Hkv]
    old = s["mass"][blk, :, t % BLOCK]
    kept = torch.where((t < s["mass_lens"][:, None])[..., None], old * 0.9375, 0.0)
    s["mass"][blk, :, t % BLOCK] = torch.where((t < s["lens"][:, None])[..., None], kept + w, old)
    return out, s["mass"]


def _plain_evict(s):
    case = s["case"]
    n, most = s["longest"], s["most"]
    t = torch.arange(n, device="cuda")
    blk = s["tables"].long()[:, t // BLOCK]
    blk = torch.where(blk < 0, s["spare"], blk)
    weight = s["mass"][blk, :, t % BLOCK].transpose(1, 2).double()          # [B, Hkv, n]
    lens, keeps = s["lens"][:, None, None], s["keeps"][:, None, None]
    recent = keeps.clamp(max=case["recent"])
    sink = torch.minimum(keeps - recent, torch.full_like(keeps, case["sink"]))
    weight = weight.masked_fill((t < sink) | (t >= lens - recent), math.inf)
    weight = weight.masked_fill(t >= lens, -math.inf)
    order = torch.sort(weight, dim=-1, descending=True, stable=True)[1][..., :most]
    j = torch.arange(order.shape[-1], device="cuda")
    kept = torch.where(j < torch.minimum(keeps, lens), order, n).sort(-1)[0]
    src = kept.transpose(1, 2)                                              # [B, most, Hkv]
    real = src < n
    st = torch.where(real, src, 0)
    b = torch.arange(case["B"], device="cuda")[:, None, None]
    g = torch.arange(case["Hkv"], device="cuda")
    dblk = torch.where(real, blk[:, :order.shape[-1], None], s["spare"])
    sblk = torch.where(real, blk[b, st], dblk)
    drow = (j % BLOCK)[None, :, None].expand_as(st)
    srow = torch.where(real, st % BLOCK, drow)
    for c in (s["k_cache"], s["v_cache"], s["mass"]):
        c[dblk, g, drow] = c[sblk, g, srow]
    kept = torch.where(kept < n, kept, -1)
    if kept.shape[-1] < most:
        kept = torch.cat([kept, kept.new_full((*kept.shape[:2], most - kept.shape[-1]), -1)], -1)
    return kept.to(torch.int32), s["k_cache"], s["v_cache"], s["mass"]


# --------------------------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rotary":
        return _exact_rotary(s)
    if case["op"] == "evict":
        return _exact_evict(s)
    return _exact_shared(s)


def _exact_rotary(s):
    case = s["case"]
    r, h = case["rot"], case["rot"] // 2
    p, base = ROTARY[case["scaling"]], BASE[case["scaling"]]
    N, F = p["original"], p["factor"]
    freq = []
    for i in range(h):
        f = (base * F ** (r / (r - 2.0)) if case["scaling"] == "ntk" else base) ** (-2.0 * i / r)
        if case["scaling"] == "linear":
            f /= F
        if case["scaling"] == "bands":
            turns = N * f / (2 * math.pi)
            if turns < p["low"]:
                f /= F
            elif turns <= p["high"]:
                w = (turns - p["low"]) / (p["high"] - p["low"])
                f = w * f + (1 - w) * f / F
        if case["scaling"] == "ramp":
            lo = max(0, math.floor(h * math.log(N / p["high"] / 2 / math.pi, base)))
            hi = min(r - 1, math.ceil(h * math.log(N / p["low"] / 2 / math.pi, base)))
            w = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = (1 - w) * f + w * f / F
        freq.append(f)
    ang = s["pos"].double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    unit = torch.polar(torch.full_like(ang, p["amplitude"]), ang)

    def turn(x):
        x = x.double().clone()
        if case["layout"] == "half":
            z = torch.complex(x[..., :h].contiguous(), x[..., h:r].contiguous()) * unit
            x[..., :h], x[..., h:r] = z.real, z.imag
        else:
            z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * unit
            x[..., 0:r:2], x[..., 1:r:2] = z.real, z.imag
        return x

    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kc[s["slots"] // BLOCK, :, s["slots"] % BLOCK] = turn(s["k"])
    vc[s["slots"] // BLOCK, :, s["slots"] % BLOCK] = s["v"].double()
    return turn(s["q"]), kc, vc


def _exact_shared(s):
    case = s["case"]
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    G = Hq // Hkv
    lens = s["lens"].tolist()
    out = torch.zeros((B, Hq, d), dtype=torch.float64, device="cuda")
    mass = s["mass"].double() if case["mass"] else None

    def gather(table, n):
        blocks = table[:-(-n // BLOCK)].long()
        kv = []
        for c in (s["k_cache"], s["v_cache"]):
            x = c[blocks].double().transpose(0, 1).reshape(Hkv, -1, d)
            kv.append(x[:, :n])
        return kv

    prefix = {p: gather(s["ptables"][p], s["plens"][p]) for p in set(s["rows"]) if p >= 0}
    for b in range(B):
        keys, values = gather(s["tables"][b], lens[b])
        at = 0
        if s["rows"][b] >= 0:
            pk, pv = prefix[s["rows"][b]]
            at = pk.shape[1]
            keys, values = torch.cat([pk, keys], 1), torch.cat([pv, values], 1)
        if keys.shape[1] == 0:
            continue
        q = s["q"][b].double().view(Hkv, G, d)
        w = torch.softmax(torch.einsum("hgd,hld->hgl", q, keys) * s["scale"], -1)
        out[b] = torch.einsum("hgl,hld->hgd", w, values).reshape(Hq, d)
        if mass is not None and lens[b]:
            t = torch.arange(lens[b], device="cuda")
            blk = s["tables"][b].long()[t // BLOCK]
            old = mass[blk, :, t % BLOCK] * 0.9375
            old[int(s["mass_lens"][b]):] = 0.0
            mass[blk, :, t % BLOCK] = old + w[:, :, at:].sum(1).t()
    return (out, mass) if mass is not None else out


def _exact_evict(s):
    case = s["case"]
    B, Hkv = case["B"], case["Hkv"]
    kept = torch.full((B, Hkv, s["most"]), -1, dtype=torch.int32)
    kc, vc, mass = s["k_cache"].double(), s["v_cache"].double(), s["mass"].double()
    for b, (L, K) in enumerate(zip(s["lens"].tolist(), s["keeps"].tolist())):
        table = s["tables"][b].long()
        t = torch.arange(L, device="cuda")
        for g in range(Hkv):
            if K < L:
                n_recent = min(case["recent"], K)
                n_sink = min(case["sink"], K - n_recent)
                mid = mass[table[t // BLOCK], g, t % BLOCK][n_sink:L - n_recent].cpu().numpy()
                best = (-mid).argsort(kind="stable")[:K - n_recent - n_sink]
                src = torch.cat([torch.arange(n_sink), torch.from_numpy(best).sort()[0] + n_sink,
                                 torch.arange(L - n_recent, L)])
            else:
                src = torch.arange(L)
            kept[b, g, :len(src)] = src.int()
            src, j = src.cuda(), torch.arange(len(src), device="cuda")
            for c in (kc, vc, mass):
                c[table[j // BLOCK], g, j % BLOCK] = c[table[src // BLOCK], g, src % BLOCK]
    return None, kc, vc, mass
