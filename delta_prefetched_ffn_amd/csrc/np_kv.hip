// Host side of the 8-bit key/value cache (np_kv_* of include/np.h): the page bookkeeping, which is
// the host's alone and exact, the checks of every call, and the launches. Nothing is enqueued and
// no state changes before every check of a call has passed.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <unordered_map>
#include <utility>
#include <vector>

#include "kv_host.hpp"

using namespace np;

namespace {

// Attention over few rows splits the key axis into workgroups for every compute unit: one each while
// a wave then has at most kFewPieces pieces (each further workgroup costs the launch a join), two
// each beyond (one's start and join hide behind the other's stream). Measured where 256 workgroups
// have 2, 4 and 63 pieces a wave: 256 workgroups 13.5, 18.5 and 216 us, 512 workgroups 20.7, 23.0 and
// 192 us, 1024 workgroups 20.7, 33.3 and 193 us.
constexpr int kCus = 256;
constexpr int kFewPieces = 16;

// Sequences of many rows (query tokens x heads of a group) may run in large tiles on the matrix units
// (k_attn_tile) instead of 16-row tiles (k_attn_rows). The first is bound by its steps of 64 tokens
// (the longest workgroup's, or all of them over the compute units), the second by the bytes and
// products of its row tiles plus a start and a join of each, and it splits the key axis where there
// are few. Microseconds, measured at 1 Ki .. 4 Ki tokens x 32 heads and at 32 .. 512 rows over 0 .. 20 Ki
// tokens: a tile's step, 256 rows x 64 tokens in row tiles, a row tile. E.g. head_dim 128, 16 bits: 4 Ki
// tokens x 32 heads 167 against 499 us; 512 rows x 8 heads over 20 Ki tokens 606 against 107 us. For
// fp32 the tiles pay up to 64 values a head (4 Ki tokens x 32 heads: 234 against 344 us); beyond, q's
// three summands leave a wave too few registers.
constexpr int kManyRows = 128;

// A launch has at most 2^32 - 1 threads along x: workgroups of k_kv_append (256 threads) and of k_attn_rows.
// (k_attn_tile's stay below for the 2^30 rows x heads a call may have.)
constexpr int64_t kMaxAppendBlocks = (int64_t)1 << 24;
constexpr int64_t kMaxRowTiles = ((int64_t)1 << 32) / (64 * kAttnWaves);
struct TileCost {
    double step, unit;
};
constexpr double kRowTileCost = 0.018;
TileCost tile_cost(int dtype, int slabs) {
    static constexpr TileCost k16[4] = {{1.9, 0.007}, {2.2, 0.020}, {4.3, 0.027}, {4.8, 0.032}};
    return dtype != NP_F32 ? k16[slabs - 1] : TileCost{3.4, 0.0113};
}

typedef std::pair<int32_t, int32_t> Move;  // page src -> dst

// Enqueues page copies (every layer); sources and destinations are disjoint.
np_status copy_pages(np_kv* kv, const std::vector<Move>& moves, hipStream_t s) {
    if (moves.empty() || kv->host_only()) return NP_OK;
    CopyArgs a;
    a.codes = static_cast<uint8_t*>(kv->desc.codes);
    a.exps = kv->desc.exps;
    a.page_bytes = kv->page_bytes;
    a.layer_bytes = kv->layer_bytes;
    a.exps_page = kv->desc.n_kv_heads * 2;
    a.exps_layer = (int64_t)kv->desc.n_pages * a.exps_page;
    a.layers = kv->desc.n_layers;
    for (size_t i = 0; i < moves.size(); i += kCopyPairs) {
        a.n = (int32_t)std::min<size_t>(kCopyPairs, moves.size() - i);
        for (int k = 0; k < a.n; ++k) {
            a.src[k] = moves[i + k].first;
            a.dst[k] = moves[i + k].second;
        }
        const hipError_t e = launch_kv_copy(a, s);
        if (e != hipSuccess) {
            kv->broken = true;
            return fail(NP_EHIP, "page copy failed: %s", hipGetErrorString(e));
        }
    }
    return NP_OK;
}

// Writes the entries that changed since the last flush, as they are now, to the device's page table.
np_status flush_table(np_kv* kv, hipStream_t s) {
    TableArgs a;
    a.table = kv->table;
    a.n = 0;
    const auto launch = [&]() -> np_status {
        const hipError_t e = a.n ? launch_kv_table(a, s) : hipSuccess;
        a.n = 0;
        if (e == hipSuccess) return NP_OK;
        kv->broken = true;
        return fail(NP_EHIP, "page table update failed: %s", hipGetErrorString(e));
    };
    for (const int32_t q : kv->stale) {
        Seq& seq = kv->seqs[q];
        const int32_t end = std::min<int32_t>(seq.stale_hi, (int32_t)seq.pages.size());
        for (int32_t i = seq.stale_lo; i < end && !kv->host_only(); ++i) {
            a.at[a.n] = q * kv->desc.max_pages + i;
            a.page[a.n] = seq.pages[i];
            if (++a.n == kTableEntries) {
                const np_status st = launch();
                if (st != NP_OK) return st;
            }
        }
        seq.stale_lo = seq.stale_hi = 0;
    }
    kv->stale.clear();
    return launch();
}

np_status check_seq(const np_kv* kv, int32_t seq, const char* what) {
    if (seq < 0 || seq >= kv->desc.max_seqs)
        return fail(NP_EINVAL, "%s %d out of range [0, %d)", what, seq, kv->desc.max_seqs);
    return NP_OK;
}

// A sequence may end inside a page only if it still holds that page: later tokens go there.
np_status check_tail(const np_kv* kv, int32_t seq, int32_t n_tokens) {
    if (n_tokens % kv->pt() && kv->seqs[seq].pages[n_tokens / kv->pt()] < 0)
        return fail(NP_EINVAL, "sequence %d has dropped the page of token %d", seq, n_tokens - 1);
    return NP_OK;
}

np_status check_desc(const np_kv_desc& D) {
    if (D.n_layers < 1 || D.n_layers > 1024) return fail(NP_EINVAL, "n_layers=%d must be in [1, 1024]", D.n_layers);
    if (D.n_kv_heads < 1 || D.n_kv_heads > 1024 || D.n_heads < 1 || D.n_heads > 4096 || D.n_heads % D.n_kv_heads)
        return fail(NP_EINVAL, "n_heads=%d must be a multiple of n_kv_heads=%d, at most 4096 and 1024", D.n_heads, D.n_kv_heads);
    if (D.head_dim < 8 || D.head_dim > kMaxHeadDim || D.head_dim % 8)
        return fail(NP_EINVAL, "head_dim=%d must be a multiple of 8 in [8, %d]", D.head_dim, kMaxHeadDim);
    if (D.page_tokens != 16 && D.page_tokens != 32 && D.page_tokens != 64 && D.page_tokens != 128)
        return fail(NP_EINVAL, "page_tokens=%d must be 16, 32, 64 or 128", D.page_tokens);
    if (D.n_pages < 1 || D.n_pages > 1 << 24) return fail(NP_EINVAL, "n_pages=%d must be in [1, 2^24]", D.n_pages);
    if (D.max_seqs < 1 || D.max_seqs > 4096) return fail(NP_EINVAL, "max_seqs=%d must be in [1, 4096]", D.max_seqs);
    if (D.max_pages < 1 || (int64_t)D.max_pages * D.page_tokens > kMaxSeqTokens)
        return fail(NP_EINVAL, "max_pages=%d must be at least 1 and hold at most 2^28 tokens", D.max_pages);
    if ((int64_t)D.max_pages * D.max_seqs > (int64_t)1 << 28)
        return fail(NP_EINVAL, "the page table (max_seqs * max_pages) must have at most 2^28 entries");
    return NP_OK;
}

int slabs_of(const np_kv_desc& D) { return (D.head_dim + kTileDims - 1) / kTileDims; }
int64_t page_bytes_of(const np_kv_desc& D) {
    return (int64_t)D.n_kv_heads * 2 * D.page_tokens * slabs_of(D) * kTileDims;
}

np_status create(const np_kv_desc* desc, np_kv** out) {
    if (!desc || !out) return fail(NP_EINVAL, "desc and out must not be NULL");
    *out = nullptr;
    const np_kv_desc& D = *desc;
    np_status st = check_desc(D);
    if (st != NP_OK) return st;
    struct Holder {
        np_kv* kv = new np_kv();
        ~Holder() { delete kv; }
    } hold;
    np_kv* const kv = hold.kv;
    kv->desc = D;
    kv->slabs = slabs_of(D);
    kv->page_shift = __builtin_ctz((unsigned)D.page_tokens);
    kv->page_bytes = page_bytes_of(D);
    kv->layer_bytes = kv->page_bytes * D.n_pages;
    kv->clear();
    kv->reserve();
    if (D.device != NP_KV_HOST) {
        if (!D.codes || !D.exps || !aligned16(D.codes) || ((uintptr_t)D.exps & 1u))
            return fail(NP_EINVAL, "codes and exps must be device pointers, 16-byte and 2-byte aligned");
        int ndev = 0;
        NP_HIP(hipGetDeviceCount(&ndev));
        if (D.device < 0 || D.device >= ndev) return fail(NP_EINVAL, "device %d out of range [0, %d)", D.device, ndev);
        DeviceGuard g(D.device);
        if (!g.ok) return fail(NP_EHIP, "hipSetDevice(%d) failed", D.device);
        if ((st = check_io_ptr(D.codes, D.device, "codes", "cache")) != NP_OK) return st;
        if ((st = check_io_ptr(D.exps, D.device, "exps", "cache")) != NP_OK) return st;
        const size_t table_bytes = (size_t)D.max_seqs * D.max_pages * sizeof(int32_t);
        const size_t part_bytes = (size_t)kMaxSharedRows * (kv->slabs * kTileDims + 2) * sizeof(float);
        if (hipMalloc((void**)&kv->table, table_bytes) != hipSuccess || hipMalloc((void**)&kv->part, part_bytes) != hipSuccess ||
            hipMalloc((void**)&kv->arrived, kMaxPartials * sizeof(uint32_t)) != hipSuccess) {
            (void)hipGetLastError();
            return fail(NP_ENOMEM, "cannot allocate the page table (%zu bytes) and scratch (%zu bytes)", table_bytes, part_bytes);
        }
        NP_HIP(attn_prepare());
        NP_HIP(hipMemset(kv->table, 0xff, table_bytes));
        NP_HIP(hipMemset(kv->arrived, 0, kMaxPartials * sizeof(uint32_t)));
        NP_HIP(hipDeviceSynchronize());
    }
    *out = kv;
    hold.kv = nullptr;
    return NP_OK;
}

np_status extend(np_kv* kv, int32_t n, const int32_t* seqs, const int32_t* n_new, hipStream_t s) {
    np_status st = check_kv(kv);
    if (st != NP_OK) return st;
    if (n < 1 || n > kMaxBatch || !seqs || !n_new)
        return fail(NP_EINVAL, "extend needs 1..%d sequences, got %d", kMaxBatch, n);
    const int pt = kv->pt();
    int64_t need = 0, rows = 0;
    std::unordered_map<int32_t, int32_t> left;  // references given up so far by copies on write
    std::vector<char> twice(kv->desc.max_seqs, 0);
    std::vector<char> cow(n, 0);
    for (int i = 0; i < n; ++i) {
        if ((st = check_seq(kv, seqs[i], "sequence")) != NP_OK) return st;
        if (twice[seqs[i]]++) return fail(NP_EINVAL, "sequence %d appears twice", seqs[i]);
        if (n_new[i] < 0 || n_new[i] > kMaxSeqTokens) return fail(NP_EINVAL, "n_new[%d]=%d must be in [0, 2^28]", i, n_new[i]);
        const Seq& q = kv->seqs[seqs[i]];
        const int64_t len = (int64_t)q.tokens + n_new[i];
        if (kv->pages_for(len) > kv->desc.max_pages)
            return fail(NP_ECAPACITY, "sequence %d: %lld tokens exceed max_pages=%d of %d", seqs[i], (long long)len, kv->desc.max_pages, pt);
        need += std::max(0, kv->pages_for(len) - (int)q.pages.size());
        if (n_new[i] > 0 && q.tokens % pt) {
            const int32_t p = q.pages[q.tokens / pt];
            if (kv->refs[p] - left[p] > 1) {
                cow[i] = 1;
                ++left[p];
                ++need;
            }
        }
        rows += n_new[i];
    }
    if (need > kv->n_free) return fail(NP_ECAPACITY, "%lld pages needed, %d free", (long long)need, kv->n_free);
    if (rows > 1 << 28) return fail(NP_EINVAL, "%lld new tokens in one call exceed 2^28", (long long)rows);

    std::vector<Move> moves;
    moves.reserve(n);
    for (int i = 0; i < n; ++i) {
        Seq& q = kv->seqs[seqs[i]];
        kv->reserve_pages(q, kv->pages_for((int64_t)q.tokens + n_new[i]));
    }
    std::optional<DeviceGuard> g;
    if ((st = make_current(kv, g)) != NP_OK) return st;

    // From here on nothing is refused. A page given up by a copy is still held by another sequence,
    // so copies read pages that nothing writes.
    kv->drop_batch();
    for (int i = 0; i < n; ++i) {
        Seq& q = kv->seqs[seqs[i]];
        kv->b_seq.push_back(seqs[i]);
        kv->b_before.push_back(q.tokens);
        kv->b_fresh.push_back(n_new[i]);
        if (cow[i]) {
            int32_t& at = q.pages[q.tokens / pt];
            const int32_t p = kv->take();
            moves.push_back({at, p});
            kv->release(at);
            at = p;
            kv->touch(seqs[i], q.tokens / pt, q.tokens / pt + 1);
        }
        q.tokens += n_new[i];
        const int32_t had = (int32_t)q.pages.size();
        while ((int)q.pages.size() < kv->pages_for(q.tokens)) q.pages.push_back(kv->take());
        kv->touch(seqs[i], had, (int32_t)q.pages.size());
    }
    if ((st = copy_pages(kv, moves, s)) != NP_OK) return st;
    return flush_table(kv, s);
}

np_status append(np_kv* kv, int32_t layer, const void* k, const void* v, int32_t dtype, const int64_t* strides, hipStream_t s) {
    np_status st = check_layer_io(kv, layer, dtype);
    if (st != NP_OK) return st;
    const np_kv_desc& D = kv->desc;
    const int64_t plain[4] = {(int64_t)D.n_kv_heads * D.head_dim, D.head_dim, (int64_t)D.n_kv_heads * D.head_dim, D.head_dim};
    const int64_t* const S = strides ? strides : plain;
    if ((st = check_rows(kv, k, S[0], S[1], dtype, "k")) != NP_OK) return st;
    if ((st = check_rows(kv, v, S[2], S[3], dtype, "v")) != NP_OK) return st;
    if (kv->host_only()) return fail(NP_ESTATE, "a bookkeeping-only cache holds no tokens");
    if ((st = check_io_ptr(k, D.device, "k", "cache")) != NP_OK) return st;
    if ((st = check_io_ptr(v, D.device, "v", "cache")) != NP_OK) return st;
    AppendArgs a;
    a.kv = kv->view();
    a.x[0] = k;
    a.x[1] = v;
    for (int i = 0; i < 2; ++i) {
        a.row_stride[i] = S[2 * i];
        a.head_stride[i] = S[2 * i + 1];
    }
    a.layer = layer;
    fill_batch(kv, a.b, [&](int i) {
        const int b = kv->b_before[i], f = kv->b_fresh[i];
        return f ? kv->pages_for((int64_t)b + f) - (b >> kv->page_shift) : 0;
    });
    if (a.b.item0[a.b.n] == 0) return NP_OK;
    if ((int64_t)a.b.item0[a.b.n] * D.n_kv_heads >= kMaxAppendBlocks)
        return fail(NP_EINVAL, "%d pages of %d heads in one call are too many", a.b.item0[a.b.n], D.n_kv_heads);
    std::optional<DeviceGuard> g;
    if ((st = make_current(kv, g)) != NP_OK) return st;
    NP_HIP(launch_kv_append(a, dtype, s));
    return NP_OK;
}

np_status attend(np_kv* kv, int32_t layer, const void* q, void* out, float* lse, int32_t dtype, const int64_t* strides,
                 float scale, int32_t window, int32_t sinks, hipStream_t s) {
    int64_t S[4], rows = 0;
    np_status st = check_attend(kv, layer, q, out, lse, dtype, strides, scale, window, sinks, S, &rows);
    if (st != NP_OK) return st;
    const np_kv_desc& D = kv->desc;
    if (rows == 0) return NP_OK;

    AttnArgs a;
    a.kv = kv->view();
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.q_row = S[0];
    a.q_head = S[1];
    a.o_row = S[2];
    a.o_head = S[3];
    a.scale2 = scale * 1.44269504088896341f;
    // Beyond the longest sequence both mean "all"; the kernels' differences then stay within 32 bits.
    window = std::min(window, 2 * kMaxSeqTokens);
    sinks = std::min(sinks, 2 * kMaxSeqTokens);
    a.window = window;
    a.sinks = sinks;
    a.layer = layer;
    a.part = kv->part;
    a.arrived = kv->arrived;
    const int group = D.n_heads / D.n_kv_heads, n = (int)kv->b_seq.size();
    if (rows * D.n_heads > 1 << 30) return fail(NP_EINVAL, "%lld rows of %d heads in one call are too many", (long long)rows, D.n_heads);
    std::optional<DeviceGuard> g;
    if ((st = make_current(kv, g)) != NP_OK) return st;
    const int tile_rows = attn_tile_rows(dtype, kv->slabs);
    const auto large = [&](int i) { return tile_rows > 0 && (int64_t)kv->b_fresh[i] * group >= kManyRows; };
    double longest = 0, steps = 0, units = 0, row_tiles = 0;
    for (int i = 0; i < n; ++i) {
        if (!large(i)) continue;
        // Steps of the first and of the last tile; those between lie between.
        const double f = kv->b_fresh[i], all_rows = f * group, seen = window ? (double)window + sinks + tile_rows / group : 1e18;
        const double last = std::min(kv->b_before[i] + f, seen) / 64 + 1;
        const double first = std::min(kv->b_before[i] + std::min(f, (double)tile_rows / group), seen) / 64 + 1;
        longest = std::max(longest, last);
        steps += std::ceil(all_rows / tile_rows) * D.n_kv_heads * (first + last) / 2;
        units += all_rows / 256 * D.n_kv_heads * (first + last) / 2;
        row_tiles += std::ceil(all_rows / kRowTile) * D.n_kv_heads;
    }
    const TileCost cost = tile_cost(dtype, kv->slabs);
    const bool pays = cost.step * std::max(longest, steps / kCus) < cost.unit * units + kRowTileCost * row_tiles;
    const auto many = [&](int i) { return pays && large(i); };
    // Pieces of a sequence's last row tile (the most of its tiles), and of all tiles together.
    const auto tiles = [&](int i) { return many(i) ? 0 : (kv->b_fresh[i] * group + kRowTile - 1) / kRowTile; };
    const auto pieces = [&](int i) {
        const int64_t len = (int64_t)kv->b_before[i] + kv->b_fresh[i];
        const int64_t span = std::min<int64_t>(kv->b_fresh[i], (kRowTile - 1) / group + 1);  // positions of a row tile
        return (window ? std::min(len, (int64_t)window + span + std::min<int64_t>(sinks, len) + kPieceTokens) : len) / kPieceTokens + 1;
    };
    int64_t all = 0;
    a.row_cap = 1;
    for (int i = 0; i < n; ++i) {
        all += pieces(i) * tiles(i) * D.n_kv_heads;
        if (tiles(i)) a.row_cap = std::max(a.row_cap, std::min(kRowTile, kv->b_fresh[i] * group));
    }
    // Pieces of a workgroup: one per wave at least, else so many that the launch is not a few workgroups
    // more than its turns hold (they would be a turn of their own).
    const int64_t most = kCus * (all > (int64_t)kCus * kAttnWaves * kFewPieces ? 2 : 1);
    const auto splits = [&](int i, int64_t per) { return (pieces(i) + per - 1) / per; };
    int64_t per = std::max<int64_t>(kAttnWaves, all / most);
    for (;; per += per / 16 + 1) {
        int64_t wgs = 0, least = 0;
        for (int i = 0; i < n; ++i) {
            wgs += tiles(i) * splits(i, per) * D.n_kv_heads;
            least += tiles(i) * D.n_kv_heads;
        }
        if (wgs <= std::max(most, least)) break;
    }
    int64_t partials = 0, row_wgs = 0;
    for (int i = 0; i < n; ++i) {
        int64_t sp = std::max<int64_t>(1, splits(i, per));
        if ((partials + tiles(i) * sp) * D.n_kv_heads > std::min(kMaxPartials, kMaxPartialRows / a.row_cap)) sp = 1;
        a.b.splits[i] = (int32_t)sp;
        a.b.part0[i] = (int32_t)partials;
        if (sp > 1) partials += tiles(i) * sp;
        row_wgs += tiles(i) * sp;
    }
    if (row_wgs >= kMaxRowTiles) return fail(NP_EINVAL, "%lld tiles of %d rows in one call are too many", (long long)row_wgs, kRowTile);
    fill_batch(kv, a.b, [&](int i) { return many(i) ? (kv->b_fresh[i] * group + tile_rows - 1) / tile_rows : 0; });
    if (a.b.item0[n] > 0) {
        a.part = nullptr;
        NP_HIP(launch_attn(a, dtype, s));
        a.part = kv->part;
    }
    if (!all) return NP_OK;
    fill_batch(kv, a.b, [&](int i) { return tiles(i) * a.b.splits[i]; });
    NP_HIP(launch_attn(a, dtype, s));
    return NP_OK;
}

np_status fork(np_kv* kv, int32_t src, int32_t dst, int32_t n_tokens, int32_t mode, hipStream_t s) {
    np_status st = check_kv(kv);
    if (st != NP_OK) return st;
    if ((st = check_seq(kv, src, "src")) != NP_OK || (st = check_seq(kv, dst, "dst")) != NP_OK) return st;
    if (src == dst || !kv->seqs[dst].pages.empty()) return fail(NP_EINVAL, "dst %d must be another, empty sequence", dst);
    if (n_tokens < 0 || n_tokens > kv->seqs[src].tokens)
        return fail(NP_EINVAL, "n_tokens=%d must be in [0, %d]", n_tokens, kv->seqs[src].tokens);
    if (mode != NP_KV_SHARE && mode != NP_KV_COPY) return fail(NP_EINVAL, "unknown mode %d", mode);
    if ((st = check_tail(kv, src, n_tokens)) != NP_OK) return st;
    const std::vector<int32_t>& from = kv->seqs[src].pages;
    const int n = kv->pages_for(n_tokens);
    if (mode == NP_KV_COPY) {
        const int64_t need = std::count_if(from.begin(), from.begin() + n, [](int32_t p) { return p >= 0; });
        if (need > kv->n_free) return fail(NP_ECAPACITY, "%lld pages needed, %d free", (long long)need, kv->n_free);
    }
    Seq& q = kv->seqs[dst];
    std::vector<Move> moves;
    if (mode == NP_KV_COPY) moves.reserve(n);
    kv->reserve_pages(q, n);
    std::optional<DeviceGuard> g;
    if (mode == NP_KV_COPY && (st = make_current(kv, g)) != NP_OK) return st;
    q.pages.assign(from.begin(), from.begin() + n);
    q.tokens = n_tokens;
    kv->drop_batch_of(dst);
    for (int32_t& p : q.pages) {
        if (p < 0) continue;
        if (mode == NP_KV_COPY) {
            moves.push_back({p, kv->take()});
            p = moves.back().second;
        } else {
            ++kv->refs[p];
        }
    }
    kv->touch(dst, 0, n);
    return copy_pages(kv, moves, s);
}

np_status adopt(np_kv* kv, int32_t seq, const int32_t* pages, int32_t n_pages, int32_t n_tokens) {
    np_status st = check_kv(kv);
    if (st != NP_OK) return st;
    if ((st = check_seq(kv, seq, "sequence")) != NP_OK) return st;
    if (!kv->seqs[seq].pages.empty()) return fail(NP_EINVAL, "sequence %d is not empty", seq);
    if (n_pages < 0 || n_pages > kv->desc.max_pages || (n_pages && !pages))
        return fail(NP_EINVAL, "n_pages=%d must be in [0, %d]", n_pages, kv->desc.max_pages);
    if (n_tokens < 0 || n_tokens > (int64_t)n_pages * kv->pt())
        return fail(NP_EINVAL, "n_tokens=%d must be in [0, %lld]", n_tokens, (long long)n_pages * kv->pt());
    std::vector<uint64_t> taken(kv->free_w.size(), 0);
    for (int i = 0; i < n_pages; ++i) {
        const int32_t p = pages[i];
        if (p == -1 && (int64_t)(i + 1) * kv->pt() <= n_tokens) continue;  // a dropped page of past tokens
        if (p < 0 || p >= kv->desc.n_pages) return fail(NP_EINVAL, "pages[%d]=%d out of range [0, %d)", i, p, kv->desc.n_pages);
        const uint64_t bit = 1ull << (p & 63);
        if (!(kv->free_w[p >> 6] & bit) || (taken[p >> 6] & bit)) return fail(NP_EINVAL, "pages[%d]=%d is in use", i, p);
        taken[p >> 6] |= bit;
    }
    Seq& q = kv->seqs[seq];
    kv->reserve_pages(q, n_pages);
    q.pages.assign(pages, pages + n_pages);
    q.tokens = n_tokens;
    kv->drop_batch_of(seq);
    for (int32_t p : q.pages)
        if (p >= 0) kv->take_page(p);
    kv->touch(seq, 0, n_pages);
    return NP_OK;
}

np_status evict(np_kv* kv, int32_t seq, int32_t window, int32_t sinks, int32_t* n_freed) {
    np_status st = check_kv(kv);
    if (st != NP_OK) return st;
    if ((st = check_seq(kv, seq, "sequence")) != NP_OK) return st;
    if (window < 1 || sinks < 0) return fail(NP_EINVAL, "window=%d must be positive and sinks=%d not negative", window, sinks);
    Seq& q = kv->seqs[seq];
    // Tokens [sinks, tokens - window] are visible to no later query: whole pages of them go.
    const int64_t end = (int64_t)q.tokens - window + 1;
    int32_t freed = 0;
    for (int64_t i = kv->pages_for(sinks); (i + 1) * kv->pt() <= end; ++i) {
        int32_t& p = q.pages[i];
        if (p < 0) continue;
        kv->release(p);
        p = -1;
        ++freed;
        kv->touch(seq, (int32_t)i, (int32_t)i + 1);
    }
    if (n_freed) *n_freed = freed;
    if (freed) kv->drop_batch_of(seq);
    return NP_OK;
}

np_status compact(np_kv* kv, int32_t* n_moved, hipStream_t s) {
    np_status st = check_kv(kv);
    if (st != NP_OK) return st;
    const int32_t live = kv->desc.n_pages - kv->n_free;
    std::vector<int32_t> to(kv->desc.n_pages, -1);
    std::vector<Move> moves;
    int32_t hole = 0;
    for (int32_t p = live; p < kv->desc.n_pages; ++p) {
        if (!kv->refs[p]) continue;
        while (kv->refs[hole]) ++hole;
        moves.push_back({p, hole});
        to[p] = hole++;
    }
    std::optional<DeviceGuard> g;
    if (!moves.empty() && (st = make_current(kv, g)) != NP_OK) return st;
    if (n_moved) *n_moved = (int32_t)moves.size();
    if (moves.empty()) return NP_OK;
    for (int32_t q = 0; q < kv->desc.max_seqs; ++q) {
        std::vector<int32_t>& pages = kv->seqs[q].pages;
        for (size_t i = 0; i < pages.size(); ++i)
            if (pages[i] >= live) {
                pages[i] = to[pages[i]];
                kv->touch(q, (int32_t)i, (int32_t)i + 1);
            }
    }
    for (const Move& m : moves) {
        kv->refs[m.second] = kv->refs[m.first];
        kv->refs[m.first] = 0;
        kv->free_w[m.second >> 6] &= ~(1ull << (m.second & 63));
        kv->free_w[m.first >> 6] |= 1ull << (m.first & 63);  // past the holes, so first_free holds
    }
    if ((st = copy_pages(kv, moves, s)) != NP_OK) return st;
    return kv->b_seq.empty() ? NP_OK : flush_table(kv, s);  // the current step goes on with the new pages
}

float e4m3_value(uint8_t b) {
    const int x = b >> 3 & 15, f = b & 7;
    const float v = (b & 127) == 127 ? NAN : x == 0 ? std::ldexp((float)f, -9) : std::ldexp((float)(8 + f), x - 10);
    return b & 128 ? -v : v;
}

np_status read_tokens(const np_kv* kv, int32_t layer, int32_t seq, int32_t first, int32_t n, float* k, float* v) {
    if (!kv) return fail(NP_EINVAL, "kv must not be NULL");
    np_status st = check_seq(kv, seq, "sequence");
    if (st != NP_OK) return st;
    if (layer < 0 || layer >= kv->desc.n_layers) return fail(NP_EINVAL, "layer %d out of range [0, %d)", layer, kv->desc.n_layers);
    const Seq& q = kv->seqs[seq];
    if (first < 0 || n < 0 || (int64_t)first + n > q.tokens)
        return fail(NP_EINVAL, "tokens [%d, %lld) out of range [0, %d)", first, (long long)first + n, q.tokens);
    if (kv->host_only()) return fail(NP_ESTATE, "a bookkeeping-only cache holds no tokens");
    const np_kv_desc& D = kv->desc;
    std::optional<DeviceGuard> g;
    if ((st = make_current(kv, g)) != NP_OK) return st;
    NP_HIP(hipDeviceSynchronize());
    const int pt = kv->pt(), hd64 = kv->slabs * kTileDims;
    std::vector<uint8_t> codes(kv->page_bytes);
    std::vector<int8_t> exps(D.n_kv_heads * 2);
    int32_t have = -2;
    for (int32_t j = first; j < first + n; ++j) {
        const int32_t page = q.pages[j / pt];
        if (page != have && page >= 0) {
            NP_HIP(hipMemcpy(codes.data(), static_cast<uint8_t*>(D.codes) + layer * kv->layer_bytes + page * kv->page_bytes,
                             codes.size(), hipMemcpyDeviceToHost));
            NP_HIP(hipMemcpy(exps.data(), D.exps + ((int64_t)layer * D.n_pages + page) * D.n_kv_heads * 2, exps.size(), hipMemcpyDeviceToHost));
        }
        have = page;
        const int t = j % pt;
        for (int h = 0; h < D.n_kv_heads; ++h)
            for (int side = 0; side < 2; ++side) {
                float* const dst = side ? v : k;
                if (!dst) continue;
                const uint8_t* const block = codes.data() + (size_t)(h * 2 + side) * pt * hd64 + (size_t)(t / 16) * kTileTokens * hd64;
                for (int d = 0; d < D.head_dim; ++d) {
                    const int t16 = t & 15, u = d & 63;
                    const int at = side ? (t16 / 4 * 16 + u / 4) * 16 + u % 4 * 4 + t16 % 4 : (u / 16 * 16 + t16) * 16 + u % 16;
                    dst[((size_t)(j - first) * D.n_kv_heads + h) * D.head_dim + d] =
                        page < 0 ? 0.0f : std::ldexp(e4m3_value(block[(size_t)(d / 64) * kTileBytes + at]), exps[h * 2 + side]);
                }
            }
    }
    return NP_OK;
}

}  // namespace

extern "C" {

np_status np_kv_bytes(const np_kv_desc* desc, int64_t* out2) {
    if (!desc || !out2) return fail(NP_EINVAL, "desc and out must not be NULL");
    const np_status st = check_desc(*desc);
    if (st != NP_OK) return st;
    out2[0] = page_bytes_of(*desc) * desc->n_pages * desc->n_layers;
    out2[1] = (int64_t)desc->n_layers * desc->n_pages * desc->n_kv_heads * 2;
    return NP_OK;
}

np_status np_kv_create(const np_kv_desc* desc, np_kv** out) {
    return guarded([&] { return create(desc, out); });
}

np_status np_kv_destroy(np_kv* kv) {
    if (!kv) return fail(NP_EINVAL, "kv must not be NULL");
    if (kv->host_only()) {
        delete kv;
        return NP_OK;
    }
    DeviceGuard g(kv->desc.device);
    CaptureGuard c;
    delete kv;  // its first hipFree waits for the device
    return NP_OK;
}

np_status np_kv_reset(np_kv* kv) {
    if (!kv) return fail(NP_EINVAL, "kv must not be NULL");
    return guarded([&] {
        kv->broken = false;
        kv->clear();
        return NP_OK;
    });
}

np_status np_kv_extend(np_kv* kv, int32_t n, const int32_t* seqs, const int32_t* n_new, void* stream) {
    return guarded([&] { return extend(kv, n, seqs, n_new, (hipStream_t)stream); });
}

np_status np_kv_append(np_kv* kv, int32_t layer, const void* k, const void* v, int32_t dtype, const int64_t* strides, void* stream) {
    return guarded([&] { return append(kv, layer, k, v, dtype, strides, (hipStream_t)stream); });
}

np_status np_kv_attend(np_kv* kv, int32_t layer, const void* q, void* out, float* lse, int32_t dtype, const int64_t* strides,
                       float scale, int32_t window, int32_t sinks, void* stream) {
    return guarded([&] { return attend(kv, layer, q, out, lse, dtype, strides, scale, window, sinks, (hipStream_t)stream); });
}

np_status np_kv_fork(np_kv* kv, int32_t src, int32_t dst, int32_t n_tokens, int32_t mode, void* stream) {
    return guarded([&] { return fork(kv, src, dst, n_tokens, mode, (hipStream_t)stream); });
}

np_status np_kv_trim(np_kv* kv, int32_t seq, int32_t n_tokens) {
    np_status st = check_kv(kv);
    if (st != NP_OK) return st;
    if ((st = check_seq(kv, seq, "sequence")) != NP_OK) return st;
    Seq& q = kv->seqs[seq];
    if (n_tokens < 0 || n_tokens > q.tokens) return fail(NP_EINVAL, "n_tokens=%d must be in [0, %d]", n_tokens, q.tokens);
    if ((st = check_tail(kv, seq, n_tokens)) != NP_OK) return st;
    while ((int)q.pages.size() > kv->pages_for(n_tokens)) {
        kv->release(q.pages.back());
        q.pages.pop_back();
    }
    q.tokens = n_tokens;
    kv->drop_batch_of(seq);
    return NP_OK;
}

np_status np_kv_free(np_kv* kv, int32_t seq) { return np_kv_trim(kv, seq, 0); }

np_status np_kv_adopt(np_kv* kv, int32_t seq, const int32_t* pages, int32_t n_pages, int32_t n_tokens) {
    return guarded([&] { return adopt(kv, seq, pages, n_pages, n_tokens); });
}

np_status np_kv_evict(np_kv* kv, int32_t seq, int32_t window, int32_t sinks, int32_t* n_freed) {
    return guarded([&] { return evict(kv, seq, window, sinks, n_freed); });
}

np_status np_kv_compact(np_kv* kv, int32_t* n_moved, void* stream) {
    return guarded([&] { return compact(kv, n_moved, (hipStream_t)stream); });
}

np_status np_kv_read_pages(const np_kv* kv, int32_t seq, int32_t* pages, int32_t cap, int32_t* n_pages, int32_t* n_tokens) {
    if (!kv || !n_pages) return fail(NP_EINVAL, "kv and n_pages must not be NULL");
    const np_status st = check_seq(kv, seq, "sequence");
    if (st != NP_OK) return st;
    const Seq& q = kv->seqs[seq];
    if (pages && cap < (int32_t)q.pages.size()) return fail(NP_EINVAL, "cap=%d is below the %zu pages", cap, q.pages.size());
    if (pages) std::copy(q.pages.begin(), q.pages.end(), pages);
    *n_pages = (int32_t)q.pages.size();
    if (n_tokens) *n_tokens = q.tokens;
    return NP_OK;
}

np_status np_kv_read_tokens(const np_kv* kv, int32_t layer, int32_t seq, int32_t first, int32_t n, float* k, float* v) {
    return guarded([&] { return read_tokens(kv, layer, seq, first, n, k, v); });
}

np_status np_kv_info(const np_kv* kv, int32_t* out4) {
    if (!kv || !out4) return fail(NP_EINVAL, "kv and out must not be NULL");
    out4[0] = kv->desc.n_pages;
    out4[1] = kv->n_free;
    out4[2] = (int32_t)std::count_if(kv->refs.begin(), kv->refs.end(), [](int32_t r) { return r > 1; });
    out4[3] = (int32_t)kv->b_seq.size();
    return NP_OK;
}

}  // extern "C"
