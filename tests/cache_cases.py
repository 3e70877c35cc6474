"""Batches of paged sequences, and the plain 64-bit definitions of the operators over them.

Rows of a pool that belong to no key hold NaN: nothing may depend on them.
Error bounds count roundings: one to bf16 is off by at most 2^-8 of the value, one
to fp32 by 2^-24, and a sum of n fp32 terms by n 2^-24 of the sum of their sizes."""
import math
from dataclasses import dataclass

import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8   # half a step of fp32 and bf16, relative


@dataclass
class Batch:
    q: torch.Tensor
    offs: torch.Tensor
    k_pages: torch.Tensor
    v_pages: torch.Tensor
    pages: torch.Tensor
    lens: torch.Tensor
    mask: torch.Tensor | None
    k: list          # per sequence [kv, Hkv, D], as stored
    v: list

    def cuda(self):
        f = lambda t: None if t is None else t.cuda()  # noqa: E731
        return Batch(f(self.q), f(self.offs), f(self.k_pages), f(self.v_pages), f(self.pages), f(self.lens),
                     f(self.mask), self.k, self.v)


def random_tree(n, g):
    seen = torch.zeros(n, n, dtype=torch.bool)
    for t in range(n):
        if t:
            seen[t] = seen[int(torch.randint(0, t, (1,), generator=g))]
        seen[t, t] = True
    return seen


def make_batch(seqs, Hq, Hkv, D, page, dtype, mask="chain", seed=0, max_pages=None, scale=1.0):
    """seqs: (keys, new tokens) of each sequence.  mask: chain, tree, empty (no new token seen), random,
    narrow (random, fewer columns than new tokens)."""
    g = torch.Generator().manual_seed(seed)
    news = [n for _, n in seqs]
    offs = torch.tensor([0] + news).cumsum(0).to(torch.int32)
    R = int(offs[-1])
    per = [-(-kv // page) for kv, _ in seqs]
    cols = max_pages or max(per + [1])
    n_pages = sum(per) + 2
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    k_pages = torch.full((n_pages, page, Hkv, D), float("nan"), dtype=dtype)
    v_pages = torch.full((n_pages, page, Hkv, D), float("nan"), dtype=dtype)
    pages = torch.full((len(seqs), cols), -7, dtype=torch.int32)   # entries past a sequence's pages are no pages
    ks, vs, used = [], [], 0
    for b, (kv, _) in enumerate(seqs):
        k = (torch.randn(kv, Hkv, D, generator=g) * scale).to(dtype)
        v = torch.randn(kv, Hkv, D, generator=g).to(dtype)
        ks.append(k)
        vs.append(v)
        for i in range(per[b]):
            pg = int(order[used])
            used += 1
            pages[b, i] = pg
            rows = k[i * page:(i + 1) * page]
            k_pages[pg, :rows.shape[0]] = rows
            v_pages[pg, :rows.shape[0]] = v[i * page:(i + 1) * page]
    m = None
    if mask != "chain":
        W = max(news + [1])
        m = torch.zeros(R, W, dtype=torch.bool)
        for b, n in enumerate(news):
            lo = int(offs[b])
            if mask == "tree":
                m[lo:lo + n, :n] = random_tree(n, g)
            elif mask in ("random", "narrow"):
                m[lo:lo + n] = torch.rand(n, W, generator=g) < 0.5   # bits past n count for nothing
        if mask == "narrow":
            m = m[:, :max(1, W // 2)].contiguous()
    q = torch.randn(R, Hq, D, generator=g).to(dtype)
    return Batch(q, offs, k_pages, v_pages, pages, torch.tensor([kv for kv, _ in seqs], dtype=torch.int32), m, ks, vs)


def visible(b, s):
    """[n, kv] bool: which keys the new tokens of sequence s see."""
    lo, hi = int(b.offs[s]), int(b.offs[s + 1])
    n, kv = hi - lo, int(b.lens[s])
    j = torch.arange(kv)[None, :] - (kv - n)      # which new token a key is
    t = torch.arange(n)[:, None]
    if b.mask is None:
        return j <= t
    m = b.mask[lo:hi].cpu()
    W = m.shape[1]
    got = torch.gather(m, 1, j.clamp(0, W - 1).expand(n, kv)) & (j < W)
    return got | (j < 0)


def attention(b):
    """(out, lse, bound of out, bound of lse) in 64 bits; the bounds for a kernel with fp32 sums whose
    weights are rounded to the storage type once."""
    R, Hq, D = b.q.shape
    Hkv = b.k_pages.shape[2]
    G = Hq // Hkv
    u_store = U16 if b.q.dtype == torch.bfloat16 else U32
    out = torch.zeros(R, Hq, D, dtype=torch.float64)
    lse = torch.full((Hq, R), -math.inf, dtype=torch.float64)
    e_out, e_lse = torch.zeros_like(out), torch.zeros(Hq, R, dtype=torch.float64)
    for s in range(len(b.k)):
        lo, hi = int(b.offs[s]), int(b.offs[s + 1])
        see = visible(b, s)
        n, kv = see.shape
        some = see.any(1)
        if not n or not kv:
            continue
        for h in range(Hq):
            q, k, v = b.q[lo:hi, h].double().cpu(), b.k[s][:, h // G].double(), b.v[s][:, h // G].double()
            x = (q @ k.T) / math.sqrt(D)
            x = x.masked_fill(~see, -math.inf)
            L = torch.logsumexp(x, 1)
            p = torch.where(some[:, None], torch.exp(x - L[:, None]), torch.zeros_like(x))
            lse[h, lo:hi] = L
            out[lo:hi, h] = p @ v
            # a score is a sum of D products (each of its own rounding) then two scalings; the exponent
            # adds a rounding of the largest score's size, the exponential 4 steps of its value
            size = ((q.abs() @ k.abs().T) / math.sqrt(D)).masked_fill(~see, 0.0).amax(1)
            e_s = (D + 6) * U32 * size + 8 * U32
            A = p @ v.abs()
            e_out[lo:hi, h] = (u_store + 2 * e_s + 2 * (kv + 16) * U32)[:, None] * A * 1.01 + u_store * out[lo:hi, h].abs() + 1e-30
            e_lse[h, lo:hi] = torch.where(some, e_s + (kv + 16) * U32 + 4 * U32 * L.abs(), torch.zeros_like(L))
    return out, lse, e_out, e_lse


def mass(b, lse, mass_in, decay, cols):
    """(gathered weight, its bound), rows with lse = -inf adding nothing; NaN where nothing is written."""
    R, Hq, D = b.q.shape
    Hkv = b.k_pages.shape[2]
    G = Hq // Hkv
    got = torch.full((len(b.k), Hkv, cols), math.nan, dtype=torch.float64)
    err = torch.zeros_like(got)
    for s in range(len(b.k)):
        lo, hi = int(b.offs[s]), int(b.offs[s + 1])
        see = visible(b, s)
        n, kv = see.shape
        for kh in range(Hkv):
            total = torch.zeros(kv, dtype=torch.float64)
            e = torch.zeros(kv, dtype=torch.float64)
            for h in range(kh * G, (kh + 1) * G):
                q, k = b.q[lo:hi, h].double().cpu(), b.k[s][:, kh].double()
                x = (q @ k.T) / math.sqrt(D)
                L = lse[h, lo:hi].double()
                p = torch.where(see & (L > -math.inf)[:, None], torch.exp(x - L[:, None]), torch.zeros_like(x))
                size = (q.abs() @ k.abs().T) / math.sqrt(D)
                e_s = (D + 6) * U32 * size + 4 * U32 * L.abs().nan_to_num(posinf=0.0)[:, None] + 8 * U32
                total += p.sum(0)
                e += (p * e_s).sum(0)
            e += (n * G + 4) * U32 * total
            if mass_in is not None:
                old = decay * mass_in[s, kh, :kv].double()
                total = total + old
                e += 2 * U32 * (old.abs() + total.abs())
            got[s, kh, :kv] = total
            err[s, kh, :kv] = e * 1.01 + 1e-30
    return got, err


def select(mass, lens, budget, first, recent):
    """positions, counts and kept mass, straight from the definition."""
    n, H, _ = mass.shape
    pos = torch.full((n, H, budget), -1, dtype=torch.int32)
    kept = torch.zeros(n, H, budget)
    counts = lens.clamp(max=budget).to(torch.int32)
    for s in range(n):
        kv = int(lens[s])
        for h in range(H):
            x = mass[s, h, :kv].tolist()
            if kv <= budget:
                keep = list(range(kv))
            else:
                free = list(range(first, kv - recent))
                value = lambda j: -math.inf if math.isnan(x[j]) else x[j] + 0.0  # noqa: E731
                # NaN below -inf; ties to the lower position
                order = sorted(free, key=lambda j: (math.isnan(x[j]), -value(j), j))
                keep = sorted(list(range(first)) + order[:budget - first - recent] + list(range(kv - recent, kv)))
            pos[s, h, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
            kept[s, h, :len(keep)] = mass[s, h, keep]
    return pos, counts, kept
