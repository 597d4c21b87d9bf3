// Host side of the attention over shared first pages (np_attend_shared of include/np.h): which runs of pages the sequences of
// the batch share, how a call's work is divided, its checks and launches. Nothing is enqueued before every check has passed.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <vector>

#include "kv_host.hpp"
#include "prefix_internal.hpp"

using namespace np;

namespace {

// A run is worth an item of its own from so many tokens on; shorter ones are read with what lies behind them.
constexpr int32_t kLeastRun = 64;
// From so many rows (new tokens x heads of a group) of a sequence on, np_kv_attend's large tiles are ahead.
constexpr int64_t kManyRows = 128;
// Microseconds, measured: a workgroup's start and end, a piece of 32 tokens of a wave (for one row tile, and for the most of
// them), the second launch, and what each partial result of a row adds to it. Against them np_kv_attend: its start, and the
// megabytes that its row tiles read in one (shared pages come from the caches there). The same for every type and head_dim: of 1,600
// random calls (2 to 100 sequences behind 200 to 25,000 tokens, head_dim 40 to 256, layers of 600 MB in turn) the slower way is
// taken, by more than 5 in 100, in 12 of a hundred: 9 that had better be shared (at worst 50 sequences behind 639 tokens, 32 heads of 64
// in fp32: 37 us for 20), 3 that had better not (at worst 16 sequences of 3 new tokens behind 1,800, 56 over 8 heads of 128 in bf16:
// 24 us for 16).
constexpr double kStart = 7.0, kNarrow = 0.75, kWide = 1.0, kJoin = 6.0, kPartial = 0.1;
constexpr double kAttendStart = 8.0, kAttendRate = 13.0;
constexpr int kCus = 256;

// How the calls with these arguments are divided; kept while the batch lasts (the layers of a step have the same).
struct Plan {
    int32_t dtype = -1, window = 0, sinks = 0;
    bool alone = false;  // np_kv_attend
    PrefixArgs args;
};
struct Plans {
    Plan plan[4];
    int next = 0;
};

// The tree of the batch's page lists: sequences whose first pages are the same are together as long as they are. Fills
// kv->order (positions in the batch of those with new tokens; those that share are neighbours) and kv->runs (a run before
// those of fewer sequences behind it).
void find_runs(np_kv* kv) {
    if (kv->runs_known) return;
    const int n = (int)kv->b_seq.size(), pt = kv->pt();
    kv->order.clear();
    kv->runs.clear();
    kv->plans.reset();
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

// Divides the batch's work: fills p.args (all but the call's addresses, layer and scale), or says that it is np_kv_attend's.
void make_plan(np_kv* kv, Plan& p, int32_t dtype, int32_t window, int32_t sinks) {
    const np_kv_desc& D = kv->desc;
    const int n = (int)kv->order.size(), group = D.n_heads / D.n_kv_heads, tiles = run_tiles(dtype, kv->slabs);
    p.alone = true;
    if (kv->runs.empty()) return;

    PrefixArgs& a = p.args;
    a.n = n;
    a.cum[0] = 0;
    a.even = kv->b_fresh[kv->order[0]];
    int64_t most_rows = 0;
    std::vector<int32_t> row0(kv->b_seq.size() + 1, 0);
    for (size_t i = 0; i < kv->b_seq.size(); ++i) row0[i + 1] = row0[i] + kv->b_fresh[i];
    a.rows = row0.back();
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
    if (most_rows >= kManyRows) return;

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
    if (found.empty()) return;

    struct Item {
        int64_t tiles, pieces, cap, splits;
        double piece;  // us of a wave
        double time() const { return kStart + piece * (double)((pieces + splits * kRunWaves - 1) / (splits * kRunWaves)); }
    };
    const auto item = [&](int64_t all_rows, int64_t tokens) {
        const bool wide = all_rows > kRowTile;
        const int64_t tile = wide ? tiles * kRowTile : kRowTile;
        return Item{(all_rows + tile - 1) / tile, tokens / kPieceTokens + 1, std::min(tile, all_rows), 1, wide ? kWide : kNarrow};
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
        work.push_back(item((int64_t)(a.cum[r.hi] - a.cum[r.lo]) * group, window ? found[k].tokens : r.t1 - x.t0));
        for (int i = r.lo; i < r.hi; ++i) {
            start[i] = r.t1;
            a.deepest[i] = (uint8_t)k;
        }
    }
    a.leaf_cap = 1;
    for (int i = 0; i < n; ++i) {
        const int64_t fresh = a.cum[i + 1] - a.cum[i], end = a.before[i] + fresh;
        const int64_t seen = window ? std::min<int64_t>(end - start[i], (int64_t)window + fresh + std::max(0, sinks - start[i])) : end - start[i];
        work.push_back(item(fresh * group, seen));
        a.leaf_cap = std::max(a.leaf_cap, (int32_t)work.back().cap);
    }
    // Pieces of a wave: what ends first, by the longest workgroup where all are there at a time, else by the sum over the
    // device and the last ones' half.
    const double slots = kCus * run_eu(dtype, kv->slabs);
    const auto divide = [&](double t) {
        for (Item& w : work) w.splits = std::max<int64_t>(1, (int64_t)std::ceil(w.pieces * w.piece / (kRunWaves * t) - 1e-9));
    };
    double best = 1e300, best_t = 0;
    for (double t = 1; t < 1e6; t *= 1.25) {
        divide(t);
        double wgs = 0, sum = 0, longest = 0, last = 0;
        int64_t part = 0, splits = 0;
        for (size_t k = 0; k < work.size(); ++k) {
            const Item& w = work[k];
            const double count = (double)(w.tiles * w.splits * D.n_kv_heads), time = w.time();
            wgs += count;
            sum += count * time;
            longest = std::max(longest, time);
            last = time;
            splits = std::max(splits, w.splits);
            part += w.tiles * w.splits * (k < (size_t)a.n_runs ? w.cap : a.leaf_cap) * D.n_kv_heads;
        }
        if (part > kMaxSharedRows) continue;
        const double est = (wgs <= slots ? longest : std::max(longest, sum / slots + last / 2)) + kJoin + kPartial * (double)splits;
        if (est < best * 0.999) {
            best = est;
            best_t = t;
        }
        if (wgs == (double)(work.size() * D.n_kv_heads)) break;
    }
    if (!best_t) return;  // more rows than partial results have room for
    double read = 0;
    for (int i = 0; i < n; ++i) {
        const int64_t fresh = a.cum[i + 1] - a.cum[i], end = a.before[i] + fresh;
        const int64_t seen = window ? std::min<int64_t>(end, (int64_t)window + fresh + sinks) : end;
        read += (double)((fresh * group + kRowTile - 1) / kRowTile * seen) * D.n_kv_heads * 2 * kv->slabs * kTileDims;
    }
    if (best > kAttendStart + read * 1e-6 / kAttendRate) return;
    divide(best_t);
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
    a.kv = kv->view();
    a.part = kv->part;
    a.window = window;
    a.sinks = sinks;
    p.alone = false;
}

np_status attend_shared(np_kv* kv, int32_t layer, const void* q, void* out, float* lse, int32_t dtype, const int64_t* strides, float scale, int32_t window,
                        int32_t sinks, hipStream_t s) {
    int64_t S[4], rows = 0;
    np_status st = check_attend(kv, layer, q, out, lse, dtype, strides, scale, window, sinks, S, &rows);
    if (st != NP_OK) return st;
    if (rows == 0) return NP_OK;
    window = std::min(window, 2 * kMaxSeqTokens);
    sinks = window ? std::min(sinks, 2 * kMaxSeqTokens) : 0;  // without a window they say nothing
    find_runs(kv);
    if (!kv->plans) kv->plans = std::make_shared<Plans>();
    Plans& plans = *static_cast<Plans*>(kv->plans.get());
    Plan* p = nullptr;
    for (Plan& x : plans.plan)
        if (x.dtype == dtype && x.window == window && x.sinks == sinks) p = &x;
    if (!p) {
        p = &plans.plan[plans.next];
        p->dtype = -1;  // until it is made
        make_plan(kv, *p, dtype, window, sinks);
        p->dtype = dtype;
        p->window = window;
        p->sinks = sinks;
        plans.next = (plans.next + 1) % 4;
    }
    if (p->alone) return np_kv_attend(kv, layer, q, out, lse, dtype, strides, scale, window, sinks, s);
    PrefixArgs& a = p->args;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.q_row = S[0];
    a.q_head = S[1];
    a.o_row = S[2];
    a.o_head = S[3];
    a.scale2 = scale * 1.44269504088896341f;
    a.layer = layer;
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
