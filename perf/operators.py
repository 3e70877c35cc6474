"""Cases and plain forms of the operators that serve from a paged KV cache.

Four operators: attention of a tree of drafted tokens over the cache (one drafted token is ordinary
decode), the attention weight each cached key gathers, the eviction that keeps the keys with the most
of it (choice, then move into other pages), and the write of new tokens' keys and values into the
pages.  `own` chooses between the plain forms below and the framework's kernels."""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"

# What each case stands for is said above it.  ctx: the longest sequence's keys, new tokens included;
# new: the most new tokens of a sequence; ragged: the sequences' lengths and token counts differ.
LISTED = [
    # one user, one token, a short conversation: launch latency
    dict(op="tree", name="tree decode 1x1", dt=BF16, seqs=1, new=1, ctx=1000, ragged=False, tree=False, hq=32, hkv=8,
         d=128, page=16),
    # a decode batch of conversations of unlike lengths, one token each: the cache's bytes
    dict(op="tree", name="tree decode batch", dt=BF16, seqs=32, new=1, ctx=16384, ragged=True, tree=False, hq=64,
         hkv=8, d=128, page=16),
    # verification of trees of up to 25 drafted tokens over medium contexts
    dict(op="tree", name="tree verify", dt=BF16, seqs=8, new=25, ctx=8000, ragged=True, tree=True, hq=64, hkv=8,
         d=128, page=64),
    # large trees over long contexts: tensor throughput
    dict(op="tree", name="tree verify large", dt=BF16, seqs=4, new=64, ctx=32768, ragged=True, tree=True, hq=64,
         hkv=8, d=128, page=128),
    # the exact fp32 path
    dict(op="tree", name="tree verify f32", dt=F32, seqs=4, new=8, ctx=4096, ragged=True, tree=True, hq=16, hkv=4,
         d=64, page=16),
    # weights gathered at every decode step of a batch
    dict(op="mass", name="mass decode batch", dt=BF16, seqs=16, new=1, ctx=16384, ragged=True, tree=False, hq=64,
         hkv=8, d=128, page=16),
    # weights of the last 64 tokens of a prompt
    dict(op="mass", name="mass window", dt=BF16, seqs=4, new=64, ctx=16000, ragged=True, tree=False, hq=32, hkv=8,
         d=128, page=64),
    # the exact fp32 path, after a verified tree
    dict(op="mass", name="mass f32", dt=F32, seqs=2, new=8, ctx=2048, ragged=True, tree=True, hq=8, hkv=4, d=64,
         page=16),
    # a batch brought back to its budget after growing past it
    dict(op="evict", name="evict batch", dt=BF16, seqs=16, ctx=6144, budget=4096, first=4, recent=512, ragged=True,
         hkv=8, d=128, page=16),
    # a long prompt cut to a small cache
    dict(op="evict", name="evict long", dt=BF16, seqs=1, ctx=131072, budget=8192, first=16, recent=1024,
         ragged=False, hkv=8, d=128, page=64),
    # one decode step of a batch
    dict(op="append", name="append decode", dt=BF16, seqs=64, new=1, ctx=4096, ragged=True, hkv=8, d=128, page=16),
    # chunks of prompts
    dict(op="append", name="append prompt", dt=BF16, seqs=4, new=8192, ctx=16384, ragged=True, hkv=8, d=128, page=64),
]


def listed():
    return [dict(c) for c in LISTED]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "mass", "evict", "append"])
    dt = rng.choice([BF16, BF16, BF16, F32])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, dt=dt, hkv=hkv, d=d, page=rng.choice([8, 16, 32, 64, 128, 256]), ragged=rng.random() < 0.8)
    if op in ("tree", "mass"):
        c["hq"] = hkv * rng.choice([1, 2, 4, 5, 7, 8])
        c["new"] = rng.choice([1, _log(rng, 1, 64)])
        c["tree"] = c["new"] > 1 and rng.random() < 0.6
        c["seqs"] = _log(rng, 1, 32)
        # at most 512K keys in all, and 2^31 scores
        most = min(32768, (1 << 19) // c["seqs"], (1 << 31) // (c["seqs"] * c["new"] * c["hq"]))
        if dt == F32:  # the fp32 path serves checks and small models
            most = min(most, 4096, (1 << 27) // (c["seqs"] * c["new"] * c["hq"]))
        c["ctx"] = _log(rng, c["new"], max(most, c["new"]))
    elif op == "evict":
        c["seqs"] = _log(rng, 1, 32)
        c["ctx"] = _log(rng, 64, 131072 // c["seqs"] if c["seqs"] < 8 else 8192)
        c["budget"] = max(8, round(c["ctx"] * rng.uniform(0.1, 0.9)))
        c["first"] = rng.randint(0, min(16, c["budget"] // 4))
        c["recent"] = rng.randint(0, c["budget"] // 2)
    else:
        c["seqs"] = _log(rng, 1, 64)
        c["new"] = _log(rng, 1, 32768 // c["seqs"])
        c["ctx"] = c["new"] + _log(rng, 1, 16384)
    return c


# ---------------------------------------------------------------------------
# sizes that follow from a case alone
# ---------------------------------------------------------------------------
def _spread(i):
    """A fixed sequence in [0, 1) without order."""
    return (0.5 + 0.6180339887498949 * i) % 1.0


def _sizes(c):
    """(keys, new tokens) of every sequence; the first has the most of both."""
    most = c.get("new", 0)
    lens, news = [], []
    for i in range(c["seqs"]):
        f = _spread(i) if c["ragged"] and i else 1.0
        news.append(max(1, round(most * (0.4 + 0.6 * f))) if most else 0)
        lens.append(max(news[-1], 1, round(c["ctx"] * (0.25 + 0.75 * f))))
    return lens, news


def _elem(c):
    return 2 if c["dt"] == BF16 else 4


def work(c):
    lens, news = _sizes(c)
    row = c["hkv"] * c["d"] * _elem(c)  # one token's keys, or values
    pages = sum(-(-n // c["page"]) for n in lens) * 4 + 8 * c["seqs"]
    if c["op"] in ("tree", "mass"):
        R, keys = sum(news), sum(lens)
        # every earlier key, and of the new ones the chain up to the row, or a tree's path (about 4)
        seen = sum((n - t) * t + (4 * t if c["tree"] else t * (t + 1) // 2) for n, t in zip(lens, news))
        q = R * c["hq"] * c["d"] * _elem(c)
        mask = R * max(news) if c["tree"] else 0
        if c["op"] == "tree":
            return {"bytes": 2 * keys * row + 2 * q + 4 * R * c["hq"] + mask + pages,
                    "flops": 4 * c["d"] * c["hq"] * seen}
        return {"bytes": keys * row + q + 4 * R * c["hq"] + 8 * keys * c["hkv"] + mask + pages,
                "flops": 2 * c["d"] * c["hq"] * seen}
    if c["op"] == "evict":
        kept = sum(min(n, c["budget"]) for n in lens)
        return {"bytes": 4 * sum(lens) * c["hkv"] + 4 * kept * row + 8 * kept * c["hkv"] + pages,
                "flops": sum(lens) * c["hkv"]}
    return {"bytes": 4 * sum(news) * row + pages, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, shape, c):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return x.to(torch.bfloat16) if c["dt"] == BF16 else x


def _pool(g, c, n_pages):
    dt = torch.bfloat16 if c["dt"] == BF16 else torch.float32
    return torch.empty((n_pages, c["page"], c["hkv"], c["d"]), device="cuda", dtype=dt).normal_(generator=g)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens, news = _sizes(c)
    per = -(-max(lens) // c["page"])
    n_pages = c["seqs"] * per + 3
    evict = c["op"] == "evict"
    more = -(-c["budget"] // c["page"]) if evict else 0
    n_pages += c["seqs"] * more
    s = {"op": c["op"], "d": c["d"], "hkv": c["hkv"], "page": c["page"], "n": c["seqs"], "L": max(lens)}
    s["k"], s["v"] = _pool(g, c, n_pages), _pool(g, c, n_pages)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    s["pages"] = order[:c["seqs"] * per].reshape(c["seqs"], per).contiguous()
    s["lens"] = _ints(lens)
    if evict:
        s["dst"] = order[c["seqs"] * per:c["seqs"] * (per + more)].reshape(c["seqs"], more).contiguous()
        s["budget"], s["first"], s["recent"] = c["budget"], c["first"], c["recent"]
        # a few keys gather much; the newest have gathered nothing yet
        u = torch.rand((c["seqs"], c["hkv"], max(lens)), generator=g, device="cuda")
        s["mass"] = (-torch.log(u.clamp_min(1e-7))) ** 3
        age = s["lens"].view(-1, 1, 1) - torch.arange(max(lens), device="cuda")
        s["mass"].masked_fill_(age <= 64, 0.0)
        return s
    offs = [0]
    for t in news:
        offs.append(offs[-1] + t)
    R = offs[-1]
    s["offs"], s["new"] = _ints(offs), max(news)
    s["row_seq"] = torch.repeat_interleave(torch.arange(c["seqs"], device="cuda"), torch.tensor(news, device="cuda"))
    s["row_t"] = torch.arange(R, device="cuda") - s["offs"].long()[s["row_seq"]]
    if c["op"] == "append":
        s["k_rows"], s["v_rows"] = _normal(g, (R, c["hkv"], c["d"]), c), _normal(g, (R, c["hkv"], c["d"]), c)
        return s
    s["hq"] = c["hq"]
    s["q"] = _normal(g, (R, c["hq"], c["d"]), c)
    s["mask"] = None
    if c["tree"]:
        # a random tree: token t hangs from one of the earlier ones, near ones more often
        W = max(news)
        seen = torch.zeros((c["seqs"], W, W), dtype=torch.bool, device="cuda")
        u = torch.rand((c["seqs"], W), generator=g, device="cuda")
        at = torch.arange(c["seqs"], device="cuda")
        for t in range(W):
            if t:
                seen[:, t] = seen[at, (t - 1 - (u[:, t] ** 2 * t).long()).clamp(0, t - 1)]
            seen[:, t, t] = True
        s["mask"] = seen[s["row_seq"], s["row_t"]].contiguous()
    if c["op"] == "mass":
        s["lse"] = _attend(s)[1].contiguous()
        s["mass"] = torch.rand((c["seqs"], c["hkv"], max(lens)), generator=g, device="cuda")
        s["out"] = torch.zeros_like(s["mass"])
        s["decay"] = 0.9375
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _cached(s, pool):
    """[sequences, keys, kv heads, d] in 32 bits, through the page table."""
    at = torch.arange(s["L"], device="cuda")
    rows = s["pages"].long()[:, at // s["page"]] * s["page"] + at % s["page"]
    return pool.reshape(-1, s["hkv"], s["d"])[rows].float()


def _scores(s):
    """Scaled scores [sequences, kv heads, new tokens x heads of a group, keys] and where they count."""
    n, G, d = s["n"], s["hq"] // s["hkv"], s["d"]
    offs, lens = s["offs"].long(), s["lens"].long()
    t = torch.arange(s["new"], device="cuda")
    count = offs[1:] - offs[:-1]
    rows = (offs[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().reshape(n, s["new"], s["hkv"], G, d).permute(0, 2, 1, 3, 4).reshape(n, s["hkv"], -1, d)
    k = _cached(s, s["k"]).permute(0, 2, 3, 1)
    x = torch.matmul(q * (1.0 / math.sqrt(d)), k)
    j = torch.arange(s["L"], device="cuda")[None, None, :]
    new = j - (lens - count)[:, None, None]  # which new token a key is
    if s["mask"] is None:
        seen = new <= t[None, :, None]
    else:
        m = s["mask"][rows]
        seen = torch.gather(m, 2, new.clamp(0, m.shape[2] - 1).expand(n, s["new"], -1)) | (new < 0)
    seen = seen & (j < lens[:, None, None]) & (t[None, :, None] < count[:, None, None])
    seen = seen[:, None, :, None, :].expand(n, 1, s["new"], G, s["L"]).reshape(n, 1, s["new"] * G, s["L"])
    return x, seen


def _rows(s, x):
    """[sequences, kv heads, new tokens x heads of a group, ...] to the stacked rows [R, heads, ...]."""
    n, G, tail = s["n"], s["hq"] // s["hkv"], x.shape[3:]
    x = x.reshape(n, s["hkv"], s["new"], G, *tail).transpose(1, 2).reshape(n, s["new"], s["hq"], *tail)
    return x[s["row_seq"], s["row_t"]]


def _attend(s):
    x, seen = _scores(s)
    x = x.masked_fill(~seen, float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    v = _cached(s, s["v"]).transpose(1, 2)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + torch.log(total))[..., 0]
    return _rows(s, o).to(s["q"].dtype), _rows(s, lse).transpose(0, 1)


def _gathered(s):
    x, seen = _scores(s)
    G = s["hq"] // s["hkv"]
    offs = s["offs"].long()
    rows = (offs[:-1, None] + torch.arange(s["new"], device="cuda")).clamp(max=s["q"].shape[0] - 1)
    lse = s["lse"].transpose(0, 1)[rows].reshape(s["n"], s["new"], s["hkv"], G).transpose(1, 2)
    p = torch.exp(x - lse.reshape(s["n"], s["hkv"], -1, 1)).masked_fill(~seen, 0.0)
    got = s["decay"] * s["mass"] + p.sum(2)
    inside = torch.arange(s["L"], device="cuda") < s["lens"].view(-1, 1, 1)
    s["out"].copy_(torch.where(inside, got, s["out"]))
    return s["out"]


def _evict(s):
    L, budget = s["L"], s["budget"]
    j = torch.arange(L, device="cuda")
    lens = s["lens"].long().view(-1, 1, 1)
    always = (j < s["first"]) | ((j >= lens - s["recent"]) & (j < lens))
    score = s["mass"].masked_fill(always, float("inf")).masked_fill(j >= lens, float("-inf"))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :budget]
    kept = order.shape[-1]
    counts = s["lens"].clamp(max=budget)
    i = torch.arange(kept, device="cuda")
    ok = i < counts.view(-1, 1, 1)
    at = torch.sort(torch.where(ok, order, torch.full_like(order, L)), dim=-1).values
    positions = torch.full((s["n"], s["hkv"], budget), -1, dtype=torch.int32, device="cuda")
    positions[..., :kept] = torch.where(ok, at, torch.full_like(at, -1)).int()
    at = at.clamp(max=L - 1)
    left = torch.zeros((s["n"], s["hkv"], budget), device="cuda")
    left[..., :kept] = torch.gather(s["mass"], 2, at).masked_fill(~ok, 0.0)
    # slot i of head h takes the kept key i; slots past a sequence's count go nowhere (a spare row behind the pool)
    src = torch.gather(s["pages"].long()[:, None, :].expand(-1, s["hkv"], -1), 2, at // s["page"]) * s["page"] + at % s["page"]
    dst = s["dst"].long()[:, i // s["page"]] * s["page"] + i % s["page"]
    head = torch.arange(s["hkv"], device="cuda").view(1, -1, 1).expand_as(src)
    dst = dst[:, None, :].expand_as(src)
    ok = ok.expand_as(src)
    for pool in (s["k"], s["v"]):
        flat = pool.reshape(-1, s["hkv"], s["d"])
        flat[dst, head] = torch.where(ok[..., None], flat[src, head], flat[dst, head])
    return {"positions": positions, "counts": counts, "mass": left, "k": s["k"], "v": s["v"]}


def _append(s):
    at = (s["lens"] - (s["offs"][1:] - s["offs"][:-1])).long()[s["row_seq"]] + s["row_t"]
    rows = s["pages"].long()[s["row_seq"], at // s["page"]] * s["page"] + at % s["page"]
    s["k"].reshape(-1, s["hkv"], s["d"])[rows] = s["k_rows"]
    s["v"].reshape(-1, s["hkv"], s["d"])[rows] = s["v_rows"]
    return {"k": s["k"], "v": s["v"]}


def run(s):
    if own:
        import ring_context_parallelism_gb300 as ra
        if s["op"] == "tree":
            out, lse = ra.tree_attn(s["q"], s["offs"], s["k"], s["v"], s["pages"], s["lens"], tree_mask=s["mask"])
            return {"out": out, "lse": lse}
        if s["op"] == "mass":
            ra.key_mass(s["q"], s["lse"], s["offs"], s["k"], s["pages"], s["lens"], s["out"], mass_in=s["mass"],
                        decay=s["decay"], tree_mask=s["mask"])
            return {"mass": s["out"]}
        if s["op"] == "evict":
            positions, counts, mass = ra.evict_select(s["mass"], s["lens"], s["budget"], n_first=s["first"],
                                                      n_recent=s["recent"])
            ra.cache_move(s["k"], s["v"], s["pages"], s["dst"], positions, counts)
            return {"positions": positions, "counts": counts, "mass": mass, "k": s["k"], "v": s["v"]}
        ra.cache_append(s["k_rows"], s["v_rows"], s["offs"], s["k"], s["v"], s["pages"], s["lens"])
        return {"k": s["k"], "v": s["v"]}
    if s["op"] == "tree":
        out, lse = _attend(s)
        return {"out": out, "lse": lse.contiguous()}
    if s["op"] == "mass":
        return {"mass": _gathered(s)}
    return _evict(s) if s["op"] == "evict" else _append(s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------
def exact(c, seed):
    if c["op"] == "append":
        return None  # copies
    s = prepare(c, seed)
    lens = s["lens"].tolist()
    if c["op"] == "evict":
        kept = torch.zeros((s["n"], s["hkv"], s["budget"]), dtype=torch.float64)
        mass = s["mass"].double().cpu()
        for b, n in enumerate(lens):
            free = list(range(s["first"], max(s["first"], n - s["recent"])))
            room = max(0, s["budget"] - (n - len(free))) if n > s["budget"] else len(free)
            for h in range(s["hkv"]):
                x = mass[b, h]
                free_x = x[free] if free else x[:0]
                best = sorted(torch.argsort(-free_x, stable=True)[:room].tolist())
                keep = list(range(min(n, s["first"]))) + [free[i] for i in best] + list(range(max(s["first"], n - s["recent"]), n))
                kept[b, h, :len(keep)] = x[keep]
        return {"positions": None, "counts": None, "mass": kept, "k": None, "v": None}
    G, d, offs = s["hq"] // s["hkv"], s["d"], s["offs"].tolist()
    out = torch.zeros((offs[-1], s["hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((s["hq"], offs[-1]), float("-inf"), dtype=torch.float64, device="cuda")
    mass = s["out"].double() if c["op"] == "mass" else None
    for b, n in enumerate(lens):
        lo, hi = offs[b], offs[b + 1]
        t = hi - lo
        pages = s["pages"][b, :-(-n // s["page"])].long()
        keys = s["k"][pages].reshape(-1, s["hkv"], d)[:n].double()
        vals = s["v"][pages].reshape(-1, s["hkv"], d)[:n].double()
        see = torch.ones((t, n), dtype=torch.bool, device="cuda")
        see[:, n - t:] = s["mask"][lo:hi, :t] if s["mask"] is not None else torch.ones(t, t, device="cuda").tril().bool()
        for h in range(s["hq"]):
            x = s["q"][lo:hi, h].double() @ keys[:, h // G].T / math.sqrt(d)
            x[~see] = float("-inf")
            if c["op"] == "mass":
                p = torch.exp(x - s["lse"][h, lo:hi].double()[:, None])
                mass[b, h // G, :n] += p.sum(0)
                continue
            lse[h, lo:hi] = torch.logsumexp(x, -1)
            out[lo:hi, h] = torch.softmax(x, -1) @ vals[:, h // G]
        if c["op"] == "mass":
            mass[b, :, :n] += s["decay"] * s["mass"][b, :, :n].double()
    return {"mass": mass} if c["op"] == "mass" else {"out": out, "lse": lse}
