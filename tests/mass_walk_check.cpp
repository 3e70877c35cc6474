// Walks the roles of the gathered-weight kernel over a batch on the CPU, CTA by CTA, with the walk and the
// rules that the kernel itself uses (csrc/mass_walk.h), and counts what breaks their order:
//   out[0]  (sequence, KV head, tile) not walked exactly once over all CTAs
//   out[1]  lse written into a set that warps of the same tile may still read: no wait for one another since the
//           last read of it
//   out[2]  row chunks given back to their producer without having been waited for
//   out[3]  row chunks waited for or given back that hold another chunk, or are not loaded
//   out[4]  places that tell a rule for out[1] from a wrong one: runs with a second tile, an odd number of runs
//           without one between them
//   out[5]  the same for out[2]: runs of resident chunks that start past what the first chunk sees
#include <vector>

#include "../ring_context_parallelism_gb300/csrc/mass_walk.h"

using ra::CacheSeq;

namespace {

struct Cta {
    const std::vector<CacheSeq>& seqs;
    const ra::MassTiles& w;
    ra::MassWalk walk;
    long long hi;
    int head, i0, i1;
    bool next() {
        return walk.next(static_cast<int>(seqs.size()), hi, w, [&](int b, CacheSeq& s) { s = seqs[b]; }, head, i0, i1);
    }
};

struct Load {
    int b, head, chunk;
    bool is(const Load& o) const { return b == o.b && head == o.head && chunk == o.chunk; }
};

// The warp that loads the row chunks.
std::vector<Load> loads(Cta c) {
    std::vector<Load> made;
    while (c.next()) {
        const CacheSeq s = c.walk.s;
        const int nch = c.w.chunks(s);
        if (c.w.resident(s)) {
            for (int x = c.w.run_chunk(s, c.i0); x < nch; ++x) made.push_back({c.walk.b, c.head, x});
        } else {
            for (int i = c.i0; i < c.i1; i += 2)
                for (int x = c.w.first_chunk(s, i); x < nch; ++x) made.push_back({c.walk.b, c.head, x});
        }
    }
    return made;
}

// The issuer of the MMAs.
void issue(Cta c, const std::vector<Load>& made, long long* out) {
    std::vector<char> waited(made.size());
    size_t qn = 0;
    auto use = [&](size_t q, const Load& want, bool wait) {
        if (q >= made.size() || !made[q].is(want)) {
            ++out[3];
            return;
        }
        if (wait)
            waited[q] = 1;
        else if (!waited[q])
            ++out[2];
    };
    while (c.next()) {
        const CacheSeq s = c.walk.s;
        const int nch = c.w.chunks(s);
        if (nch == 0) continue;
        const bool resident = c.w.resident(s);
        const int c0 = resident ? c.w.run_chunk(s, c.i0) : 0;
        for (int i = c.i0; i < c.i1; i += 2)
            for (int x = c.w.first_chunk(s, i); x < nch; ++x) {
                const Load want{c.walk.b, c.head, x};
                use(resident ? qn + x - c0 : qn, want, true);
                if (!resident) use(qn++, want, false);
            }
        if (resident)
            for (int x = c0; x < nch; ++x) use(qn++, {c.walk.b, c.head, x}, false);
    }
    out[3] += qn != made.size();
}

// The warps of tile t of the pairs.
void weigh(Cta c, int t, long long* out) {
    ra::LseSets sets;
    long long waits = 0, read[2][ra::kMassResident];
    for (auto& set : read)
        for (auto& r : set) r = -1;
    int turn = 0, without = 0;
    bool before = false;
    while (c.next()) {
        const CacheSeq s = c.walk.s;
        const int nch = c.w.chunks(s);
        if (nch > 0) {
            if (c.i0 + t < c.i1) {
                out[4] += before && (without & 1);
                before = true;
                without = 0;
            } else {
                ++without;
            }
        }
        const bool resident = c.w.resident(s);
        const int set = sets.take(nch, c.i0, c.i1, t);
        int held = 0;
        for (int i = c.i0 + t; i < c.i1; i += 2)
            for (int x = c.w.first_chunk(s, i - t); x < nch; ++x) {
                const int buf = resident ? x : turn & 1;
                if (!resident || !((held >> x) & 1)) {
                    out[1] += read[set][buf] == waits;
                    ++waits;
                    ++turn;
                    held |= 1 << (x & 31);
                }
                read[set][buf] = waits;
            }
    }
}

}  // namespace

extern "C" void mass_walk_check(int n_seqs, const int* kv, const int* n, int heads, int rpt, int tree, int ctas,
                                long long* out) {
    for (int i = 0; i < 6; ++i) out[i] = 0;
    std::vector<CacheSeq> seqs;
    const ra::MassTiles w{heads, rpt, tree != 0};
    long long total = 0;
    std::vector<std::vector<int>> walked;
    for (int b = 0, lo = 0; b < n_seqs; lo += n[b++]) {
        seqs.push_back({lo, n[b], kv[b]});
        total += w.head(seqs[b]) * heads;
        walked.emplace_back(w.tiles(seqs[b]) * heads);
    }
    const int active = static_cast<int>(total < ctas ? (total < 1 ? 1 : total) : ctas);
    const long long q = total / active, rem = total % active;
    for (int k = 0; k < active; ++k) {
        const long long lo = k * q + (k < rem ? k : rem), hi = lo + q + (k < rem ? 1 : 0);
        if (lo >= hi) continue;
        long long before = 0, wh = 0;
        int b = 0;
        for (;; before += wh * heads, ++b)
            if (lo < before + (wh = w.head(seqs[b])) * heads) break;
        Cta c{seqs, w, {seqs[b], b, 0, 0, 0}, hi, 0, 0, 0};
        c.walk.a = before + w.locate(seqs[b], wh, lo - before, c.walk.head, c.walk.i);
        for (Cta d = c; d.next();) {
            const CacheSeq s = d.walk.s;
            for (int i = d.i0; i < d.i1; ++i) ++walked[d.walk.b][d.head * w.tiles(s) + i];
            out[5] += w.chunks(s) > 0 && w.resident(s) && w.first_chunk(s, d.i0) > 0;
        }
        issue(c, loads(c), out);
        for (int t = 0; t < 2; ++t) weigh(c, t, out);
    }
    for (auto& seq : walked)
        for (int x : seq) out[0] += x != 1;
}
