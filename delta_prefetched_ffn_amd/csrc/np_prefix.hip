// Host side of the attention over shared first pages (np_attend_shared of include/np.h): which runs of pages the sequences of
// the batch share, how a call's work is divided, its checks and launches. Nothing is enqueued before every check has passed.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>
#include <vector>

#include "kv_host.hpp"
#include "prefix_internal.hpp"

using namespace np;

namespace {

// A run is worth an item of its own from so many tokens on; shorter ones are read with what lies behind them.
constexpr int32_t kLeastRun = 64;
// Bytes of keys and values that a call must not read again for the second launch to pay.
constexpr double kLeastSaved = 0;
// From so many rows (new tokens x heads of a group) of a sequence on, np_kv_attend's large tiles are ahead.
constexpr int64_t kManyRows = 128;
// Pieces of 32 tokens that a workgroup takes at least.
constexpr int64_t kLeastPieces = 2 * kRunWaves;

// The tree of the batch's page lists: sequences whose first pages are the same are together as long as they are. Fills
// kv->order (positions in the batch of those with new tokens; those that share are neighbours) and kv->runs (a run before
// those of fewer sequences behind it).
void find_runs(np_kv* kv) {
    if (kv->runs_known) return;
    const int n = (int)kv->b_seq.size(), pt = kv->pt();
    kv->order.clear();
    kv->runs.clear();
    for (int i = 0; i < n; ++i)
        if (kv->b_fresh[i] > 0) kv->order.push_back(i);
    const auto pages = [&](int i) -> const std::vector<int32_t>& { return kv->seqs[kv->b_seq[i]].pages; };
    const auto columns = [&](int i) { return kv->b_before[i] / pt; };  // whole pages of earlier tokens: others may hold new ones
    struct Span {
        int lo, hi, from;  // of the order; pages in front of `from` are the same
    };
    std::vector<Span> todo;
    if (kv->order.size() > 1) todo.push_back({0, (int)kv->order.size(), 0});
    while (!todo.empty()) {
        const Span g = todo.back();
        todo.pop_back();
        int32_t* const o = kv->order.data();
        int same = columns(o[g.lo]);
        for (int i = g.lo + 1; i < g.hi && same > g.from; ++i) {
            const int most = std::max(std::min(same, columns(o[i])), g.from);
            const int32_t *const a = pages(o[g.lo]).data(), *const b = pages(o[i]).data();
            same = (int)(std::mismatch(a + g.from, a + most, b + g.from).first - a);
        }
        const int at = std::max(same, g.from);
        if (at > g.from) kv->runs.push_back({g.lo, g.hi, g.from * pt, at * pt});
        // Those with the same next page become neighbours; those that end here stand in front.
        const auto next = [&](int i) { return columns(i) > at ? (int64_t)pages(i)[at] : INT64_MIN; };
        std::sort(o + g.lo, o + g.hi, [&](int a, int b) { return next(a) != next(b) ? next(a) < next(b) : a < b; });
        for (int i = g.lo, j; i < g.hi; i = j) {
            for (j = i + 1; j < g.hi && next(o[j]) == next(o[i]);) ++j;
            if (j - i > 1 && next(o[i]) != INT64_MIN) todo.push_back({i, j, at});
        }
    }
    std::sort(kv->runs.begin(), kv->runs.end(), [](const SharedRun& a, const SharedRun& b) { return a.t0 < b.t0 || (a.t0 == b.t0 && a.lo < b.lo); });
    kv->runs_known = true;
}

// Tokens of [t0, t1) that are held and that a row at position pos sees.
int64_t visible(const np_kv* kv, int seq, int32_t t0, int32_t t1, int64_t pos, int32_t window, int32_t sinks) {
    const std::vector<int32_t>& pages = kv->seqs[seq].pages;
    const int64_t lo = window ? pos - window + 1 : 0;
    int64_t got = 0;
    for (int32_t c = t0 / kv->pt(); c < t1 / kv->pt(); ++c)
        if (pages[c] >= 0 && ((int64_t)(c + 1) * kv->pt() > lo || (int64_t)c * kv->pt() < sinks)) got += kv->pt();
    return got;
}

np_status attend_shared(np_kv* kv, int32_t layer, const void* q, void* out, float* lse, int32_t dtype, const int64_t* strides, float scale, int32_t window,
                        int32_t sinks, hipStream_t s) {
    int64_t S[4], rows = 0;
    np_status st = check_attend(kv, layer, q, out, lse, dtype, strides, scale, window, sinks, S, &rows);
    if (st != NP_OK) return st;
    const auto alone = [&] { return np_kv_attend(kv, layer, q, out, lse, dtype, strides, scale, window, sinks, s); };
    if (rows == 0) return NP_OK;
    window = std::min(window, 2 * kMaxSeqTokens);
    sinks = std::min(sinks, 2 * kMaxSeqTokens);
    find_runs(kv);
    const np_kv_desc& D = kv->desc;
    const int n = (int)kv->order.size(), group = D.n_heads / D.n_kv_heads, tiles = run_tiles(dtype, kv->slabs);
    if (kv->runs.empty()) return alone();

    PrefixArgs a;
    a.n = n;
    a.cum[0] = 0;
    a.even = kv->b_fresh[kv->order[0]];
    int64_t most_rows = 0;
    std::vector<int32_t> row0(kv->b_seq.size() + 1, 0);
    for (size_t i = 0; i < kv->b_seq.size(); ++i) row0[i + 1] = row0[i] + kv->b_fresh[i];
    for (int i = 0; i < n; ++i) {
        const int b = kv->order[i];
        a.seq[i] = (uint16_t)kv->b_seq[b];
        a.before[i] = kv->b_before[b];
        a.row0[i] = row0[b];
        a.cum[i + 1] = a.cum[i] + kv->b_fresh[b];
        a.deepest[i] = kNoRun;
        if (kv->b_fresh[b] != a.even) a.even = 0;
        most_rows = std::max<int64_t>(most_rows, (int64_t)kv->b_fresh[b] * group);
    }
    if (most_rows >= kManyRows) return alone();

    // The runs that pay most, as they lie one behind the other: a run starts where the chosen one in front of it ends.
    struct Candidate {
        SharedRun run;
        int64_t tokens;
    };
    std::vector<Candidate> found;
    for (const SharedRun& r : kv->runs) {
        int64_t pos = a.before[r.lo];
        for (int i = r.lo; i < r.hi; ++i) pos = std::min<int64_t>(pos, a.before[i]);
        const int64_t tokens = visible(kv, a.seq[r.lo], r.t0, r.t1, pos, window, sinks);
        if (tokens >= kLeastRun) found.push_back({r, tokens});
    }
    const auto gain = [](const Candidate& c) { return (c.run.hi - c.run.lo - 1) * c.tokens; };
    if (found.size() > kMaxRuns) {
        std::sort(found.begin(), found.end(), [&](const Candidate& x, const Candidate& y) {
            return gain(x) != gain(y) ? gain(x) > gain(y) : x.run.t0 != y.run.t0 ? x.run.t0 < y.run.t0 : x.run.lo < y.run.lo;
        });
        found.resize(kMaxRuns);
        std::sort(found.begin(), found.end(), [](const Candidate& x, const Candidate& y) { return x.run.t0 != y.run.t0 ? x.run.t0 < y.run.t0 : x.run.lo < y.run.lo; });
    }
    double saved = 0;
    for (const Candidate& c : found) saved += (double)gain(c) * D.n_kv_heads * 2 * kv->slabs * kTileDims;
    if (found.empty() || saved < kLeastSaved) return alone();

    // Work, in pieces of 32 tokens of one tile; a wide tile's piece counts as kWidePiece narrow ones'.
    struct Item {
        int64_t tiles, pieces, weight, cap, splits;
    };
    const auto item = [&](int64_t all_rows, int64_t tokens) {
        const bool wide = all_rows > kRowTile;
        const int64_t tile = wide ? tiles * kRowTile : kRowTile;
        return Item{(all_rows + tile - 1) / tile, tokens / kPieceTokens + 1, wide ? tiles / 2 : 1, std::min(tile, all_rows), 1};
    };
    std::vector<Item> work;
    a.n_runs = (int)found.size();
    std::vector<int32_t> start(n, 0);
    for (int k = 0; k < a.n_runs; ++k) {
        const SharedRun& r = found[k].run;
        PrefixRun& x = a.run[k];
        x.t0 = start[r.lo];
        x.t1 = r.t1;
        x.s0 = (uint8_t)r.lo;
        x.s1 = (uint8_t)r.hi;
        work.push_back(item((int64_t)(a.cum[r.hi] - a.cum[r.lo]) * group, std::max<int64_t>(found[k].tokens, window ? 0 : r.t1 - x.t0)));
        for (int i = r.lo; i < r.hi; ++i) {
            start[i] = r.t1;
            a.deepest[i] = (uint8_t)k;
        }
    }
    a.leaf_cap = 1;
    for (int i = 0; i < n; ++i) {
        const int64_t fresh = a.cum[i + 1] - a.cum[i], end = a.before[i] + fresh;
        const int64_t seen = window ? std::min<int64_t>(end - start[i], (int64_t)window + fresh + (sinks > start[i] ? sinks - start[i] : 0)) : end - start[i];
        work.push_back(item(fresh * group, seen));
        a.leaf_cap = std::max(a.leaf_cap, (int32_t)work.back().cap);
    }
    int64_t all = 0;
    for (const Item& w : work) all += w.tiles * w.pieces * w.weight * D.n_kv_heads;
    // A workgroup's share: a turn of the device for all, or several where each is long.
    const int64_t most = all > (int64_t)kRunSlots * kRunWaves * 32 ? 2 * kRunSlots : kRunSlots;
    int64_t wgs = 0, part = 0;
    for (int64_t per = std::max<int64_t>(kLeastPieces, all / most);; per += per / 8 + 1) {
        int64_t least = 0;
        wgs = part = 0;
        bool one = true;
        for (size_t k = 0; k < work.size(); ++k) {
            Item& w = work[k];
            w.splits = std::min<int64_t>(std::max<int64_t>(1, (w.pieces * w.weight + per - 1) / per), 65535);
            wgs += w.tiles * w.splits * D.n_kv_heads;
            least += w.tiles * D.n_kv_heads;
            part += w.tiles * w.splits * (k < (size_t)a.n_runs ? w.cap : a.leaf_cap) * D.n_kv_heads;
            one &= w.splits == 1;
        }
        if ((wgs <= std::max(most, least) && part <= kMaxSharedRows) || one) break;
    }
    if (part > kMaxSharedRows) return alone();

    a.kv = kv->view();
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.q_row = S[0];
    a.q_head = S[1];
    a.o_row = S[2];
    a.o_head = S[3];
    a.part = kv->part;
    a.scale2 = scale * 1.44269504088896341f;
    a.window = window;
    a.sinks = sinks;
    a.layer = layer;
    a.rows = (int32_t)rows;
    int32_t items = 0, parts = 0;
    for (int k = 0; k < a.n_runs; ++k) {
        a.run[k].item0 = items;
        a.run[k].part0 = parts;
        a.run[k].splits = (uint16_t)work[k].splits;
        items += (int32_t)(work[k].tiles * work[k].splits);
        parts += (int32_t)(work[k].tiles * work[k].splits * work[k].cap);
    }
    a.leaf_item = items;
    a.leaf_part = parts;
    a.item0[0] = 0;
    for (int i = 0; i < n; ++i) {
        const Item& w = work[a.n_runs + i];
        a.splits[i] = (uint16_t)w.splits;
        a.item0[i + 1] = a.item0[i] + (int32_t)(w.tiles * w.splits);
    }
    std::optional<DeviceGuard> g;
    if ((st = make_current(kv, g)) != NP_OK) return st;
    NP_HIP(launch_prefix(a, dtype, s));
    return NP_OK;
}

}  // namespace

extern "C" {

np_status np_attend_shared(np_kv* kv, int32_t layer, const void* q, void* out, float* lse, int32_t dtype, const int64_t* strides, float scale, int32_t window,
                           int32_t sinks, void* stream) {
    return guarded([&] { return attend_shared(kv, layer, q, out, lse, dtype, strides, scale, window, sinks, (hipStream_t)stream); });
}

}  // extern "C"
