"""Measured cases of decoding with drafted tokens: attention of a tree of drafted tokens over the
paged cache, pages copied (forks, a pool that moves), the accepted path moved to the front of the
drafted tokens' slots, and rotary positions with several axes.

``run`` with ``own`` false is the plain form (elementary torch operations in 32 bits); with ``own``
true it makes the calls a user makes.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one chat verifies a handful of drafted tokens: latency
        dict(name="tree_one", op="tree", B=1, Hq=8, Hkv=2, d=64, dtype="bf16", nlo=8, nhi=8, llo=500,
             lhi=500, chain=0, hollow=0, seed=1),
        # a small ragged batch, trees of different sizes, some rows with one token only
        dict(name="tree_chat16", op="tree", B=16, Hq=32, Hkv=8, d=128, dtype="bf16", nlo=1, nhi=26,
             llo=1, lhi=2600, chain=0, hollow=0, seed=2),
        # a full ragged batch with large trees
        dict(name="tree_ragged64", op="tree", B=64, Hq=32, Hkv=8, d=128, dtype="bf16", nlo=33, nhi=64,
             llo=1, lhi=4096, chain=0, hollow=0, seed=3),
        # one very long context, an odd tree
        dict(name="tree_long131k", op="tree", B=1, Hq=32, Hkv=4, d=128, dtype="bf16", nlo=61, nhi=61,
             llo=131011, lhi=131011, chain=0, hollow=0, seed=4),
        # chunks of prompts beside decoding rows: chains of 1 to 1023 tokens behind what is cached
        dict(name="tree_chunks8", op="tree", B=8, Hq=32, Hkv=8, d=128, dtype="bf16", nlo=1, nhi=1023,
             llo=0, lhi=7000, chain=1, hollow=0, seed=5),
        # 32 bits, empty contexts and nodes that see nothing among them
        dict(name="tree_f32", op="tree", B=24, Hq=16, Hkv=8, d=64, dtype="f32", nlo=1, nhi=16, llo=0,
             lhi=513, chain=0, hollow=1, seed=6),
        # forks of a few sequences: their last, half-filled pages
        dict(name="copy_forks16", op="copy", pools=2, blocks=64, pairs=16, Hkv=8, d=128, dtype="bf16"),
        # the pages of a pool that is made smaller, every layer's keys and values
        dict(name="copy_pool", op="copy", pools=16, blocks=2304, pairs=1023, Hkv=8, d=128,
             dtype="bf16"),
        # the accepted tokens of a few small trees
        dict(name="accept_few", op="accept", pools=2, B=3, Hkv=2, d=64, dtype="f32", nlo=5, nhi=16,
             alo=0, ahi=4, llo=1, lhi=100, seed=7),
        # the accepted tokens of a full batch in every layer
        dict(name="accept_64x32", op="accept", pools=64, B=64, Hkv=8, d=128, dtype="bf16", nlo=33,
             nhi=64, alo=1, ahi=12, llo=1, lhi=64, seed=8),
        # a decode step of a batch whose tokens have time, height and width
        dict(name="axes_step256", op="axes", T=256, Hq=32, Hkv=8, d=128, dtype="bf16",
             sections="16,24,24", order="blocked", ladder="shared", layout="half", scaling="plain"),
        # the patches of a video's frames, pairs dealt to the axes in turn
        dict(name="axes_video16k", op="axes", T=16384, Hq=32, Hkv=8, d=128, dtype="bf16",
             sections="24,20,20", order="cyclic", ladder="shared", layout="half", scaling="linear"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "copy", "accept", "axes"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "copy":
        pools, pairs = 2 * _spread(rng, 1, 16), _spread(rng, 1, 2000)
        pairs = max(1, min(pairs, 16000 // pools))
        return dict(op=op, pools=pools, blocks=2 * pairs + _spread(rng, 1, 500), pairs=pairs, Hkv=Hkv,
                    d=d, dtype=dtype)
    if op == "accept":
        n = _spread(rng, 2, 64)
        return dict(op=op, pools=2 * _spread(rng, 1, 32), B=_spread(rng, 1, 64), Hkv=Hkv, d=d,
                    dtype=dtype, nlo=max(1, n // 2), nhi=n, alo=rng.choice([0, 1]),
                    ahi=max(2, n // rng.choice([2, 4, 8])), llo=rng.choice([0, 1]),
                    lhi=_spread(rng, 1, 64), seed=rng.randrange(1 << 20))
    if op == "axes":
        half = d // 2
        parts = rng.choice([[1], [half // 2, half // 4], [half // 4, half // 4 + 2, half // 4 - 2],
                            [half // 4, half // 8 * 3, half // 8 * 3], [5, 6, 7],
                            [half // 8, half // 8, half // 4, half // 4]])
        return dict(op=op, T=_spread(rng, 1, 12000), Hq=Hkv * rng.choice([1, 2, 4]), Hkv=Hkv, d=d,
                    dtype=dtype, sections=",".join(map(str, parts)),
                    order=rng.choice(["blocked", "cyclic"]), ladder=rng.choice(["shared", "own"]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["plain", "linear"]))
    G = rng.choice([1, 2, 4, 8])
    B = _spread(rng, 1, 64)
    chain = rng.choice([0, 0, 1])
    n = _spread(rng, 1, min(600, 2000 // B + 1) if chain else 100)
    # the plain form's scores stay below 2 GB, float32 products below those of the chunks
    most = min(16000, (50000000 if dtype == "f32" else 500000000) // (B * n * G * Hkv))
    return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, dtype=dtype, nlo=max(1, n // 3), nhi=n,
                llo=rng.choice([0, 1]), lhi=_spread(rng, 1, max(2, min(most, 400000 // B))),
                chain=chain, hollow=rng.choice([0, 0, 1]) if not chain else 0,
                seed=rng.randrange(1 << 20))


def _sizes(case):
    """Cached tokens and nodes of every row (a function of the case)."""
    rng = random.Random(case["seed"])
    cached = [rng.randint(case["llo"], case["lhi"]) for _ in range(case["B"])]
    nodes = [rng.randint(case["nlo"], case["nhi"]) for _ in range(case["B"])]
    cached[-1], nodes[-1] = case["lhi"], case["nhi"]
    return cached, nodes


def _trees(case):
    """Per node of all rows the set of the row's nodes that it sees, as a whole number of bits:
    its ancestors and itself (a chain: all before it).  In a hollow case some see nothing."""
    rng = random.Random(case["seed"] + 1)
    rows = []
    for n in _sizes(case)[1]:
        seen = []
        for i in range(n):
            up = 0 if i == 0 else seen[i - 1] if case["chain"] else seen[rng.randint(i // 3, i - 1)]
            seen.append(up | 1 << i)
        if case["hollow"]:
            seen = [0 if rng.random() < 0.2 else s for s in seen]
        rows.append(seen)
    return rows


def _accepted(case):
    """Accepted nodes of every row, ascending: the root first, then nodes of lower levels."""
    rng = random.Random(case["seed"] + 2)
    paths = []
    for n in _sizes(case)[1]:
        a = min(rng.randint(case["alo"], case["ahi"]), (n + 1) // 2)
        paths.append([0][:a] + sorted(rng.sample(range(a, n), max(a - 1, 0))))
    return paths


def work(case):
    e, d, Hkv = ESIZE[case["dtype"]], case["d"], case["Hkv"]
    if case["op"] == "copy":
        return {"bytes": 2 * case["pools"] * case["pairs"] * Hkv * BLOCK * d * e, "flops": 0}
    if case["op"] == "accept":
        moved = sum(sum(j != p for j, p in enumerate(path)) for path in _accepted(case))
        return {"bytes": max(1, 2 * case["pools"] * moved * Hkv * d * e), "flops": 0}
    if case["op"] == "axes":
        rows = case["T"] * (case["Hq"] + 2 * Hkv)
        axes = case["sections"].count(",") + 1
        return {"bytes": 2 * rows * d * e + (4 * axes + 8) * case["T"], "flops": 3 * rows * d}
    cached, nodes = _sizes(case)
    T = sum(nodes)
    pairs = sum(c * n for c, n in zip(cached, nodes))
    if case["chain"]:
        pairs += sum(n * (n + 1) // 2 for n in nodes)
    else:
        pairs += sum(bin(s).count("1") for row in _trees(case) for s in row)
    b = 2 * (sum(cached) + T) * Hkv * d * e + 2 * T * case["Hq"] * d * e
    return {"bytes": b, "flops": 4 * d * case["Hq"] * pairs}


# --------------------------------------------------------------------------- inputs
def _gen(seed, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1009 + k)
    return g


def _normal(shape, dtype, seed, k):
    return torch.randn(shape, generator=_gen(seed, k), device="cuda", dtype=DTYPES[dtype])


def _tables(lens, seed):
    """Scattered block tables [rows, most] (int32, -1 padded) for lens tokens a row, over a pool of
    1.25 times the blocks; its size, and a block that belongs to nobody."""
    need = np.array([-(-n // BLOCK) for n in lens], np.int64)
    blocks = int(need.sum())
    n = blocks + max(1, blocks // 4)
    free = np.random.RandomState(seed % (1 << 31)).permutation(n).astype(np.int32)
    width = max(1, int(need.max()))
    j = np.arange(width)
    at = np.cumsum(need)[:, None] - need[:, None] + j
    table = np.where(j < need[:, None], free[np.minimum(at, n - 1)], -1)
    return n, torch.from_numpy(table.astype(np.int32)).cuda(), int(free[-1])


def prepare(case, seed):
    return {"tree": _prepare_tree, "copy": _prepare_copy, "accept": _prepare_accept,
            "axes": _prepare_axes}[case["op"]](case, seed)


def _starts(nodes):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)).cuda()


def _prepare_tree(case, seed):
    Hq, Hkv, d, dt = case["Hq"], case["Hkv"], case["d"], case["dtype"]
    cached, nodes = _sizes(case)
    lens = [c + n for c, n in zip(cached, nodes)]
    n, table, spare = _tables(lens, seed)
    T = sum(nodes)
    s = dict(case=case, scale=1.0 / math.sqrt(d), spare=spare, longest=max(lens), widest=max(nodes),
             tables=table, lens=torch.tensor(lens, dtype=torch.int32).cuda(), starts=_starts(nodes),
             mask=None, q=_normal((T, Hq, d), dt, seed, 1),
             k_cache=_normal((n, Hkv, BLOCK, d), dt, seed, 2),
             v_cache=_normal((n, Hkv, BLOCK, d), dt, seed, 3))
    if not case["chain"]:
        words = -(-max(nodes) // 32)
        raw = b"".join(x.to_bytes(4 * words, "little") for row in _trees(case) for x in row)
        s["mask"] = torch.from_numpy(np.frombuffer(raw, np.int32).reshape(T, words).copy()).cuda()
    if own:
        from paged_kv_decode_10_gb300 import binding
        s["out"] = torch.empty_like(s["q"])
        s["args"] = binding.make_tree_args(s["q"], s["k_cache"], s["v_cache"], table, s["lens"],
                                           s["starts"], s["scale"], s["out"], mask=s["mask"])
    return s


def _prepare_copy(case, seed):
    pool = _normal((case["pools"], case["blocks"], case["Hkv"], BLOCK, case["d"]), case["dtype"], seed, 1)
    order = np.random.RandomState(seed % (1 << 31)).permutation(case["blocks"]).astype(np.int32)
    order = torch.from_numpy(order).cuda()
    s = dict(case=case, pool=pool, src=order[:case["pairs"]].contiguous(),
             dst=order[case["pairs"]:2 * case["pairs"]].contiguous())
    if own:
        from paged_kv_decode_10_gb300 import binding
        s["args"] = binding.make_copy_args(list(pool), s["src"], s["dst"])
    return s


def _prepare_accept(case, seed):
    cached, nodes = _sizes(case)
    lens = [c + n for c, n in zip(cached, nodes)]
    n, table, spare = _tables(lens, seed)
    paths = _accepted(case)
    most = max(1, max(map(len, paths)))
    path = np.array([p + [-1] * (most - len(p)) for p in paths], np.int32)
    s = dict(case=case, spare=spare, tables=table, starts=_starts(nodes),
             lens=torch.tensor(lens, dtype=torch.int32).cuda(), path=torch.from_numpy(path).cuda(),
             counts=torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda(),
             pool=_normal((case["pools"], n, case["Hkv"], BLOCK, case["d"]), case["dtype"], seed, 1))
    if own:
        from paged_kv_decode_10_gb300 import binding
        s["args"] = binding.make_accept_args(list(s["pool"]), table, s["lens"], s["starts"], s["path"],
                                             s["counts"])
    return s


FACTOR = {"plain": 1.0, "linear": 4.0}
BASE = 1000000.0


def _prepare_axes(case, seed):
    T, Hq, Hkv, d, dt = case["T"], case["Hq"], case["Hkv"], case["d"], case["dtype"]
    sections = [int(x) for x in case["sections"].split(",")]
    qkv = _normal((T, Hq + 2 * Hkv, d), dt, seed, 1)   # one projection's output: q, k, v side by side
    rng = np.random.RandomState(seed % (1 << 31))
    # frames of 18 x 32 patches behind a text of some length; the first axis is time
    t = np.arange(T) + rng.randint(0, 50000)
    pos = np.stack([t // 576, t // 32 % 18, t % 32] + [t % 7])[:len(sections)] + rng.randint(0, 1 << 16)
    n = -(-T // BLOCK) + 3
    slots = rng.permutation(n * BLOCK)[:T].astype(np.int64)
    s = dict(case=case, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], sections=sections,
             pos=torch.from_numpy(pos.astype(np.int32)).cuda(), slots=torch.from_numpy(slots).cuda(),
             k_cache=_normal((n, Hkv, BLOCK, d), dt, seed, 2),
             v_cache=_normal((n, Hkv, BLOCK, d), dt, seed, 3))
    if own:
        from paged_kv_decode_10_gb300 import binding
        rot = binding.Rotary(d, rot_dim=2 * sum(sections), layout=case["layout"],
                             scaling=case["scaling"], base=BASE, factor=FACTOR[case["scaling"]],
                             sections=sections, order=case["order"], ladder=case["ladder"])
        s["q_out"] = torch.empty((T, Hq, d), dtype=DTYPES[dt], device="cuda")
        s["args"] = binding.make_rotary_args(rot, s["q"], s["k"], s["v"], s["pos"], q_out=s["q_out"],
                                             slot_mapping=s["slots"], k_cache=s["k_cache"],
                                             v_cache=s["v_cache"])
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        from paged_kv_decode_10_gb300 import binding
        if op == "tree":
            binding.decode_attn_tree_args(s["args"])
            return s["out"]
        if op == "copy":
            binding.copy_blocks_args(s["args"])
            return s["pool"]
        if op == "accept":
            binding.accept_nodes_args(s["args"])
            return s["pool"]
        binding.rotary_append_args(s["args"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    return {"tree": _plain_tree, "copy": _plain_copy, "accept": _plain_accept,
            "axes": _plain_axes}[op](s)


def _plain_tree(s):
    case = s["case"]
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    G, n, w = Hq // Hkv, s["longest"], s["widest"]
    t = torch.arange(n, device="cuda")
    blk = s["tables"].long()[:, t // BLOCK]
    blk = torch.where(blk < 0, s["spare"], blk)
    k, v = (c[blk, :, t % BLOCK].float().transpose(1, 2) for c in (s["k_cache"], s["v_cache"]))
    starts = s["starts"].long()
    count = starts[1:] - starts[:-1]
    base = s["lens"].long() - count
    i = torch.arange(w, device="cuda")
    there = i < count[:, None]                                           # [B, w]
    at = torch.where(there, starts[:-1, None] + i, 0)
    q = (s["q"].float() * s["scale"]).view(-1, Hkv, G, d)[at]            # [B, w, Hkv, G, d]
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, w * G, d)
    j = t - base[:, None]                                                # token's node, [B, n]
    if s["mask"] is None:
        sees = j[:, None] <= i[:, None]                                  # [B, w, n]
    else:
        words = s["mask"][at]                                            # [B, w, words]
        word = (j // 32).clamp(0, words.shape[-1] - 1)[:, None].expand(B, w, n)
        bit = (words.gather(2, word) >> (j % 32).int()[:, None]) & 1
        sees = (j < 0)[:, None] | (bit != 0)
    sees = sees & (t < s["lens"][:, None])[:, None]
    sees = sees[:, None, :, None].expand(B, 1, w, G, n).reshape(B, 1, w * G, n)
    score = (q @ k.transpose(-1, -2)).masked_fill_(~sees, -math.inf)
    m = score.amax(-1, keepdim=True)
    p = score.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p @ v).masked_fill_(l == 0, 0.0) / torch.where(l > 0, l, 1.0)
    o = o.view(B, Hkv, w, G, d).permute(0, 2, 1, 3, 4)[there]            # [T, Hkv, G, d]
    return o.reshape(-1, Hq, d).to(s["q"].dtype)


def _plain_copy(s):
    s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
    return s["pool"]


def _plain_accept(s):
    starts = s["starts"].long()
    base = s["lens"].long() - (starts[1:] - starts[:-1])
    j = torch.arange(s["path"].shape[1], device="cuda")
    real = j < s["counts"][:, None]
    src = base[:, None] + torch.where(real, s["path"].long(), 0)
    dst = base[:, None] + torch.where(real, j, 0)
    table = s["tables"].long()

    def slot(t):   # (what is not real goes from the spare block to itself)
        b = table.gather(1, (t // BLOCK).clamp(max=table.shape[1] - 1))
        return torch.where(real, b, s["spare"]), torch.where(real, t % BLOCK, 0)

    sb, sr = slot(src)
    db, dr = slot(dst)
    s["pool"][:, db, :, dr] = s["pool"][:, sb, :, sr]
    return s["pool"]


def _axis_of(sections, order):
    """Axis of every pair, and its number among the axis' pairs."""
    a = np.concatenate([np.full(n, i) for i, n in enumerate(sections)])
    k = np.concatenate([np.arange(n) for n in sections])
    if order == "cyclic":   # dealt to the axes in turn, as long as they have pairs
        by = np.lexsort((a, k))
        a, k = a[by], k[by]
    return a, k


def _plain_axes(s):
    case = s["case"]
    sections, half, dt = s["sections"], sum(s["sections"]), DTYPES[case["dtype"]]
    axis, number = _axis_of(sections, case["order"])
    if case["ladder"] == "own":
        f = BASE ** (-number / np.array(sections)[axis])
    else:
        f = BASE ** (-np.arange(half) / half)
    f = torch.from_numpy(f / FACTOR[case["scaling"]]).cuda()
    theta = s["pos"].double()[torch.from_numpy(axis).cuda()].t() * f      # [T, half]
    cos, sin = theta.cos().float()[:, None], theta.sin().float()[:, None]

    def turn(x):
        y = x.float()
        x1, x2 = (y[..., :half], y[..., half:2 * half]) if case["layout"] == "half" else (
            y[..., 0:2 * half:2], y[..., 1:2 * half:2])
        z = [x1 * cos - x2 * sin, x2 * cos + x1 * sin]
        z = torch.cat(z, -1) if case["layout"] == "half" else torch.stack(z, -1).flatten(-2)
        return torch.cat([z, y[..., 2 * half:]], -1).to(dt)

    blk, row = s["slots"] // BLOCK, s["slots"] % BLOCK
    s["k_cache"][blk, :, row] = turn(s["k"])
    s["v_cache"][blk, :, row] = s["v"]
    return turn(s["q"]), s["k_cache"], s["v_cache"]


# --------------------------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "tree":
        out = torch.zeros((s["q"].shape[0], case["Hq"], case["d"]), dtype=torch.float64, device="cuda")
        G, at = case["Hq"] // case["Hkv"], 0
        for b, (c, seen) in enumerate(zip(_sizes(case)[0], _trees(case))):
            n = len(seen)
            blocks = s["tables"][b, :-(-(c + n) // BLOCK)].long()
            sees = np.ones((n, c + n), bool)
            sees[:, c:] = [[x >> j & 1 for j in range(n)] for x in seen]
            sees = torch.from_numpy(sees).cuda()[:, None]
            for g in range(case["Hkv"]):
                k, v = (x[blocks, g].double().flatten(0, 1)[:c + n] for x in (s["k_cache"], s["v_cache"]))
                q = s["q"][at:at + n, g * G:(g + 1) * G].double()
                score = torch.einsum("nhd,ld->nhl", q, k) * s["scale"]
                weight = torch.softmax(score.masked_fill(~sees, -math.inf), -1)
                out[at:at + n, g * G:(g + 1) * G] = torch.einsum(
                    "nhl,ld->nhd", torch.nan_to_num(weight), v)   # (a node that sees nothing: zeros)
            at += n
        return out
    if case["op"] == "copy":
        pool = s["pool"].double()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            pool[:, b] = pool[:, a]
        return pool
    if case["op"] == "accept":
        pool = s["pool"].double()
        for b, (c, path) in enumerate(zip(_sizes(case)[0], _accepted(case))):
            table = s["tables"][b].tolist()
            for j, i in enumerate(path):
                src, dst = c + i, c + j
                pool[:, table[dst // BLOCK], :, dst % BLOCK] = pool[:, table[src // BLOCK], :, src % BLOCK]
        return pool
    left = list(s["sections"])
    axis = []
    while sum(left):
        for a in range(len(left)):
            take = min(left[a], 1 if case["order"] == "cyclic" else left[a])
            axis += [a] * take
            left[a] -= take
    half, freq = len(axis), []
    for i, a in enumerate(axis):
        k, m = (axis[:i].count(a), s["sections"][a]) if case["ladder"] == "own" else (i, half)
        freq.append(math.exp(-math.log(BASE) * k / m) / FACTOR[case["scaling"]])
    ang = s["pos"].double()[torch.tensor(axis).cuda()].t() * torch.tensor(freq, dtype=torch.float64).cuda()
    unit = torch.polar(torch.ones_like(ang), ang)[:, None]

    def turn(x):
        x = x.double().clone()
        at = (slice(0, half), slice(half, 2 * half)) if case["layout"] == "half" else (
            slice(0, 2 * half, 2), slice(1, 2 * half, 2))
        z = torch.complex(x[..., at[0]].contiguous(), x[..., at[1]].contiguous()) * unit
        x[..., at[0]], x[..., at[1]] = z.real, z.imag
        return x

    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kc[s["slots"] // BLOCK, :, s["slots"] % BLOCK] = turn(s["k"])
    vc[s["slots"] // BLOCK, :, s["slots"] % BLOCK] = s["v"].double()
    return turn(s["q"]), kc, vc
