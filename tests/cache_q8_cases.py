"""Batches of paged sequences in an 8-bit cache, and the plain 64-bit definitions over them.

Rows of a pool that belong to no key hold NaN codes and scale bytes that mean infinity: nothing may depend on
them."""
import math

import torch

from cache_cases import attention, make_batch

E4M3 = torch.float8_e4m3fn
TABLE = torch.arange(127, dtype=torch.uint8).view(E4M3).double()   # the codes' values, 0 to 448


def scale_bytes(rows):
    """The byte of every row [...] of rows [..., D]: the least power of two >= 2^-126 with max <= 448 scale."""
    most = rows.double().abs().amax(-1)
    e = torch.ones(most.shape, dtype=torch.int64)
    for _ in range(254):
        e = torch.where(most > 448.0 * torch.exp2(e.double() - 127), e + 1, e)
    return e.to(torch.uint8)


def codes(rows, bytes_):
    """The nearest codes to rows / scale, ties to even, by trying them all."""
    y = rows.double() / torch.exp2(bytes_.double() - 127)[..., None]
    up = torch.searchsorted(TABLE, y.abs().clamp(max=448.0)).clamp(1, 126)
    lo, hi = TABLE[up - 1], TABLE[up]
    to_hi = hi - y.abs()
    to_lo = y.abs() - lo
    at = torch.where((to_hi < to_lo) | ((to_hi == to_lo) & (up % 2 == 0)), up, up - 1)
    return (at + torch.where(torch.signbit(rows), 128, 0)).to(torch.uint8)


def value(code_bytes, bytes_):
    scale = torch.where(bytes_ == 0, 0.0, torch.exp2(bytes_.double() - 127))
    return code_bytes.view(E4M3).double() * scale[..., None]


class Batch8:
    """make_batch's sequences with their keys and values in 8 bits; k and v: their values in 64 bits."""

    def __init__(self, seqs, Hq, Hkv, D, page, dtype, mask="chain", seed=0, max_pages=None, scale=1.0, edit=None):
        b = make_batch(seqs, Hq, Hkv, D, page, torch.float32, mask, seed, max_pages, scale)
        b.q = b.q.to(dtype)
        if edit:
            edit(b)
        self.base = b
        n = b.k_pages.shape[0]
        self.pools = [torch.full((n, page, Hkv, D), 0x7F, dtype=torch.uint8) for _ in range(2)]
        self.scales = [torch.full((n, Hkv, page), 0xFF, dtype=torch.uint8) for _ in range(2)]
        for s in range(len(seqs)):
            for pool, scales, rows in ((self.pools[0], self.scales[0], b.k), (self.pools[1], self.scales[1], b.v)):
                e = scale_bytes(rows[s])
                c = codes(rows[s], e)
                for i in range(-(-rows[s].shape[0] // page)):
                    pg, part = int(b.pages[s, i]), slice(i * page, (i + 1) * page)
                    m = c[part].shape[0]
                    pool[pg, :m] = c[part]
                    scales[pg, :, :m] = e[part].T
                rows[s] = value(c, e)
        self.k, self.v = b.k, b.v

    def args(self, dev="cuda"):
        b = self.base
        return (b.q.to(dev), b.offs.to(dev), *(p.view(E4M3).to(dev) for p in self.pools), *(s.to(dev) for s in self.scales),
                b.pages.to(dev), b.lens.to(dev))

    def mask(self, dev="cuda"):
        return None if self.base.mask is None else self.base.mask.to(dev)


def attention_q8(b8):
    """(out, lse, bound of out, bound of lse): those of the attention over the cache's values, whose count of roundings
    holds (a score's scaling by its key's scale is one of them), and for bf16 queries what their two 8-bit parts and
    the weights' three leave out.

    Queries: a row is brought to a largest value in [128, 256); its first part keeps 4 bits, the second takes what is
    left of its 8, exactly but for the second part's least step of 2^-9: off by at most 2^-10 / 128 of the row's
    largest.  Weights: rounded to fp16 (2^-11 at most) and, with few rows, to three parts of 3 bits (the last of what two
    cut off, 2^-9 of the weight at most), together less than the 2^-8 that one rounding to bf16 is counted with.
    Below the least steps: a weight times its value's scale over the largest scale is off by 2^-17 2^-10 of a reference
    that is at most the row's largest weight (few rows; with many, 2^-25 2^-7, and the fp16 value by 2^-25), where the
    value's code is at most 448: for n keys n 2^-27 448 of the largest scale's unit, and 448 units are at most twice the
    sequence's largest value."""
    b = b8.base
    out, lse, e_out, e_lse = attention(b)
    if b.q.dtype != torch.bfloat16:
        return out, lse, e_out, e_lse
    R, Hq, D = b.q.shape
    Hkv = b.k_pages.shape[2]
    for s in range(len(b.k)):
        lo, hi = int(b.offs[s]), int(b.offs[s + 1])
        if hi == lo or not b.k[s].shape[0]:
            continue
        for h in range(Hq):
            k, v = b.k[s][:, h // (Hq // Hkv)], b.v[s][:, h // (Hq // Hkv)]
            left_out = 2.0 ** -17 * b.q[lo:hi, h].double().abs().amax(-1)
            e_s = left_out * k.abs().sum(-1).amax() / math.sqrt(D)
            some = lse[h, lo:hi] > -math.inf
            least = v.shape[0] * 2.0 ** -26 * b.v[s].abs().amax()
            e_out[lo:hi, h] += (2 * e_s[:, None] * v.abs().amax(0) + least) * some[:, None]
            e_lse[h, lo:hi] += e_s * some
    return out, lse, e_out, e_lse
