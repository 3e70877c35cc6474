// mass_walk.h -- which key tiles and row chunks a CTA of the gathered-weight kernel
// (key_mass_tc.cu) meets, shared by its roles and by host checks of their order.
//
// A sequence's keys are cut into tiles of kMassTile keys, its new tokens into chunks of
// rpt tokens.  The tiles of the batch, end to end over (sequence, KV head), are cut into
// ranges of equal weight; a CTA walks the tiles that start inside its range, in runs of
// consecutive tiles of one (sequence, KV head).
#pragma once

#include "ra_walk.h"

namespace ra {

// One sequence of the batch; n = 0 if it has no rows or breaks a rule.
struct CacheSeq {
    int lo;  // first stacked row
    int n;   // new tokens
    int kv;  // keys in the cache, new tokens included
};

// a / b for a, b >= 0: in 32 bits where that is enough (a third of the latency).
RA_HD long long quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return a / b;
}

constexpr int kMassTile = 128;     // keys of a tile
constexpr int kMassResident = 2;   // row chunks that stay in shared memory for a whole run; more are streamed again
constexpr int kMassOverhead = 1;   // weight of a tile beyond its chunks

// Weight of the key tiles of one KV head: the row chunks a tile meets plus kMassOverhead.
struct MassTiles {
    int heads, rpt;
    bool tree;
    RA_HD int chunks(const CacheSeq& s) const { return (s.n + rpt - 1) / rpt; }
    RA_HD bool resident(const CacheSeq& s) const { return chunks(s) <= kMassResident; }
    RA_HD int tiles(const CacheSeq& s) const { return (s.kv + kMassTile - 1) / kMassTile; }
    // first chunk with a row that sees tile i
    RA_HD int first_chunk(const CacheSeq& s, int i) const {
        const int jn = i * kMassTile - (s.kv - s.n);
        return tree || jn <= 0 || s.n == 0 ? 0 : jn / rpt;
    }
    // First chunk that a run of resident chunks from tile i0 on loads: the first one it meets.  An earlier one would
    // be given back without anyone having waited for it, so that the next load into its place, or the CTA's end,
    // could come before it has landed.
    RA_HD int run_chunk(const CacheSeq& s, int i0) const { return first_chunk(s, i0); }
    // leading tiles that meet every chunk
    RA_HD int uniform(const CacheSeq& s) const {
        const int all = tiles(s);
        const int reach = s.kv - s.n + rpt;  // keys that the first chunk sees
        if (tree || s.n <= rpt) return all;
        return reach < 1 ? 0 : clampi((reach - 1) / kMassTile + 1, 0, all);
    }
    RA_HD int tile(const CacheSeq& s, int i) const { return chunks(s) - first_chunk(s, i) + kMassOverhead; }
    RA_HD long long head(const CacheSeq& s) const {
        const int u = uniform(s), all = tiles(s);
        long long w = static_cast<long long>(u) * (chunks(s) + kMassOverhead);
        for (int i = u; i < all; ++i) w += tile(s, i);
        return w;
    }
    // Whole tiles from tile i on, of weight w0 each, until `left` of weight is reached: at most n.
    RA_HD static int whole(long long left, int w0, int n) {
        const long long k = quotient(left + w0 - 1, w0);
        return k < n ? static_cast<int>(k) : n;
    }
    // The first tile that starts at weight x of the sequence or after it (in its KV head), and the weight before it.
    RA_HD long long locate(const CacheSeq& s, long long wh, long long x, int& h, int& i) const {
        h = static_cast<int>(quotient(x, wh));
        long long a = wh * h;
        const int all = tiles(s), w0 = chunks(s) + kMassOverhead;
        i = whole(x - a, w0, uniform(s));
        a += static_cast<long long>(i) * w0;
        while (i < all && a < x) a += tile(s, i++);
        return a;
    }
};

// Runs of consecutive tiles of one (sequence, KV head) that start inside the CTA's range.
struct MassWalk {
    CacheSeq s;
    int b, head, i;
    long long a;   // weight before tile i
    // Tiles [i0, i1) of head h of sequence b, up to weight `hi`; load(b, s) reads a sequence.
    template <class Load>
    RA_HD bool next(int n_seqs, long long hi, const MassTiles& w, Load load, int& h, int& i0, int& i1) {
        for (;;) {
            if (b >= n_seqs || a >= hi) return false;
            const int all = w.tiles(s);
            if (i < all) break;
            i = 0;
            if (all == 0 || ++head >= w.heads) {
                head = 0;
                if (++b < n_seqs) load(b, s);
            }
        }
        const int u = w.uniform(s), all = w.tiles(s), w0 = w.chunks(s) + kMassOverhead;
        h = head;
        i0 = i;
        if (i < u) {
            const int k = MassTiles::whole(hi - a, w0, u - i);
            i += k;
            a += static_cast<long long>(k) * w0;
        }
        while (i < all && a < hi) a += w.tile(s, i++);
        i1 = i;
        return true;
    }
};

// A run's tiles are walked in pairs; the warps of tile t of the pairs keep the lse of the run's rows in one of two
// sets and wait for one another between writing it and reading it.  The sets change with the runs in which these
// warps have a tile, so between two uses of a set lies a use of the other one, and with it a wait.  (A run of one
// tile leaves the second warps without any: if it changed their set too, a warp could write a set that slower ones
// still read.)
struct LseSets {
    int runs = 0;
    // The set for a run of tiles [i0, i1) over `chunks` row chunks.
    RA_HD int take(int chunks, int i0, int i1, int t) {
        const int set = runs & 1;
        if (chunks > 0 && i0 + t < i1) ++runs;
        return set;
    }
};

}  // namespace ra
