// kv_stub.cpp, with the launches of the attention over shared pages, the rotary positions and the products with 4-bit weights:
// compiled together with their host sides (np_prefix.hip, np_rope.hip, np_w4.hip, np_kv.hip) by tests/test_ops_host.py.
#include "kv_stub.cpp"

#include <algorithm>
#include <cstring>
#include <set>

#include "prefix_internal.hpp"
#include "rope_internal.hpp"
#include "w4_internal.hpp"

namespace {
np::PrefixArgs g_prefix;
np::RopeArgs g_rope;
np::RopeAppendArgs g_append;
np::W4Args g_w4;
long g_prefix_calls = 0, g_attend_calls = 0;
int g_prefix_dtype = 0;
std::string g_why;

// What the kernels of k_prefix.hip make of the last call: every (row, token) once, partial results apart and in bounds.
const char* check_prefix() {
    using namespace np;
    const PrefixArgs& a = g_prefix;
    const int group = a.kv.n_heads / a.kv.n_kv, tiles = run_tiles(g_prefix_dtype, a.kv.slabs);
    const auto bad = [&](const char* what, int x, int y) {
        g_why = std::string(what) + " (" + std::to_string(x) + ", " + std::to_string(y) + ")";
        return g_why.c_str();
    };
    if (a.n_runs < 1 || a.n_runs > kMaxRuns) return bad("runs", a.n_runs, 0);
    const int rows = a.cum[a.n] * group;
    // per row: the token ranges of its parts, in order, and the partial rows they leave
    std::vector<std::vector<std::pair<int, int>>> seen(rows);
    std::set<int64_t> used;
    const auto part = [&](int64_t at) { return at >= 0 && (at + 1) * a.kv.n_kv <= kMaxSharedRows && used.insert(at).second; };
    for (int k = 0; k < a.n_runs; ++k) {
        const PrefixRun& r = a.run[k];
        const int end = k + 1 < a.n_runs ? a.run[k + 1].item0 : a.leaf_item;
        const int all = (a.cum[r.s1] - a.cum[r.s0]) * group, tile = all <= kRowTile ? kRowTile : tiles * kRowTile, cap = std::min(tiles * kRowTile, all);
        const int n_tiles = (all + tile - 1) / tile;
        if (r.s1 - r.s0 < 2 || r.t0 >= r.t1 || r.t0 % (1 << a.kv.page_shift) || r.t1 % (1 << a.kv.page_shift)) return bad("run", k, r.t1);
        if (end - r.item0 != n_tiles * r.splits) return bad("items of run", k, end - r.item0);
        for (int t = 0; t < n_tiles; ++t)
            for (int s = 0; s < r.splits; ++s)
                for (int x = 0; x < std::min(tile, all - t * tile); ++x)
                    if (!part(r.part0 + (int64_t)(t * r.splits + s) * cap + x)) return bad("partial row of run", k, t);
        for (int x = 0; x < all; ++x) seen[a.cum[r.s0] * group + x].push_back({r.t0, r.t1});
        for (int s = r.s0; s < r.s1; ++s) {
            if (r.t1 > a.before[s]) return bad("new tokens in run", k, s);
            for (int p = r.t0 >> a.kv.page_shift; p < r.t1 >> a.kv.page_shift; ++p) {
                const int64_t i = (int64_t)a.seq[s] * a.kv.max_pages + p, j = (int64_t)a.seq[r.s0] * a.kv.max_pages + p;
                if (g_table[i] != g_table[j]) return bad("other page in run", k, s);
            }
        }
    }
    for (int s = 0; s < a.n; ++s) {
        const int fresh = a.cum[s + 1] - a.cum[s], all = fresh * group, tile = all <= kRowTile ? kRowTile : tiles * kRowTile, n_tiles = (all + tile - 1) / tile;
        if (fresh < 1 || (a.even && fresh != a.even)) return bad("new tokens", s, fresh);
        if (a.item0[s + 1] - a.item0[s] != n_tiles * a.splits[s] || a.splits[s] < 1) return bad("items", s, a.splits[s]);
        for (int i = a.item0[s]; i < a.item0[s + 1]; ++i)
            for (int x = 0; x < std::min(tile, all - (i - a.item0[s]) / a.splits[s] * tile); ++x)
                if (x >= a.leaf_cap || !part(a.leaf_part + (int64_t)i * a.leaf_cap + x)) return bad("partial row", s, i);
        const int from = a.deepest[s] == kNoRun ? 0 : a.run[a.deepest[s]].t1;
        for (int x = 0; x < all; ++x) seen[a.cum[s] * group + x].push_back({from, a.before[s] + x / group + 1});
    }
    for (int r = 0; r < rows; ++r) {
        int at = 0;
        std::sort(seen[r].begin(), seen[r].end());
        for (const auto& p : seen[r]) {
            if (p.first != at) return bad("gap or overlap at row and token", r, at);
            at = p.second;
        }
    }
    return "";
}
}  // namespace

extern "C" {
long stub_prefix_calls() { return g_prefix_calls; }
const char* stub_check_prefix() { return check_prefix(); }
int stub_prefix_runs() { return g_prefix.n_runs; }
long stub_rope_items() { return (long)g_rope.rows * ((np::rope_groups(g_rope.rope.hd, g_rope.x[0].heads + g_rope.x[1].heads) + g_rope.per - 1) / g_rope.per); }
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) { return hipSuccess; }
}

namespace np {
hipError_t launch_prefix(const PrefixArgs& a, int dtype, hipStream_t) {
    g_prefix = a;
    g_prefix_dtype = dtype;
    const hipError_t e = launch((uint64_t)(a.leaf_item + a.item0[a.n]) * a.kv.n_kv * 64 * kRunWaves);
    if (e == hipSuccess) ++g_prefix_calls;
    return e;
}
hipError_t launch_rope(const RopeArgs& a, int, hipStream_t) {
    g_rope = a;
    return launch((uint64_t)(stub_rope_items() + 3) / 4 * 256);
}
hipError_t launch_rope_append(const RopeAppendArgs& a, int, hipStream_t) {
    g_append = a;
    return launch((uint64_t)append_grid(a) * append_threads(a.kv.page_shift, a.kv.hd, a.kv.slabs));
}
hipError_t launch_w4_pack(const W4PackArgs&, hipStream_t) { return launch(256); }
hipError_t launch_w4(const W4Args& a, int, hipStream_t) {
    g_w4 = a;
    return launch((uint64_t)((a.rows + 63) / 64) * ((a.w.out_tiles + 63) / 64 * 8) * 512);
}
hipError_t w4_prepare() { return hipSuccess; }
}  // namespace np
