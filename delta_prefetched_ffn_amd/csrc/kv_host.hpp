// One key/value cache as the library's host files see it: its page books, and the checks that its calls
// share (np_kv.hip has the np_kv_* calls; others that work on a cache use these).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>
#include <optional>
#include <vector>

#include "kv_internal.hpp"
#include "np.h"
#include "np_host.hpp"

namespace np {

struct Seq {
    std::vector<int32_t> pages;  // -1: dropped
    int32_t tokens = 0;
    int32_t stale_lo = 0, stale_hi = 0;  // entries that the device's page table does not have yet
};

// Tokens [t0, t1) (whole pages, all earlier than the new ones) that the sequences order[lo .. hi) of the batch share.
struct SharedRun {
    int32_t lo, hi, t0, t1;
};

}  // namespace np

struct np_kv {
    np_kv_desc desc{};
    int slabs = 0, page_shift = 0;
    int64_t page_bytes = 0, layer_bytes = 0;
    std::vector<int32_t> refs;      // sequences that hold each page
    std::vector<uint64_t> free_w;   // bit set: free
    size_t first_free = 0;          // no word before it has a bit set
    int32_t n_free = 0;
    std::vector<np::Seq> seqs;
    std::vector<int32_t> stale;     // sequences with such entries
    std::vector<int32_t> b_seq, b_before, b_fresh;  // the current batch (np_kv_extend); empty: none
    // What the batch's sequences share, worked out by the first call that asks (np_prefix.hip).
    bool runs_known = false;
    std::vector<int32_t> order;     // positions in the batch
    std::vector<np::SharedRun> runs;
    std::shared_ptr<void> plans;    // and how its calls are divided
    bool broken = false;            // a launch failed in the middle of a call
    int32_t* table = nullptr;
    float* part = nullptr;
    uint32_t* arrived = nullptr;

    bool host_only() const { return desc.device == NP_KV_HOST; }
    int pt() const { return desc.page_tokens; }
    int pages_for(int64_t tokens) const { return (int)((tokens + pt() - 1) >> page_shift); }

    int32_t take() {  // the free page with the lowest number (the caller has counted them)
        while (!free_w[first_free]) ++first_free;
        const int32_t p = (int32_t)(first_free * 64 + __builtin_ctzll(free_w[first_free]));
        take_page(p);
        return p;
    }
    void take_page(int32_t p) {
        free_w[p >> 6] &= ~(1ull << (p & 63));
        refs[p] = 1;
        --n_free;
    }
    void release(int32_t p) {
        if (p < 0 || --refs[p] > 0) return;
        free_w[p >> 6] |= 1ull << (p & 63);
        first_free = std::min(first_free, (size_t)p >> 6);
        ++n_free;
    }
    // Entries [lo, hi) of a sequence have changed.
    void touch(int32_t seq, int32_t lo, int32_t hi) {
        np::Seq& q = seqs[seq];
        if (lo >= hi) return;
        if (q.stale_lo == q.stale_hi) {
            stale.push_back(seq);
            q.stale_lo = lo;
            q.stale_hi = hi;
        } else {
            q.stale_lo = std::min(q.stale_lo, lo);
            q.stale_hi = std::max(q.stale_hi, hi);
        }
    }
    void drop_batch_of(int32_t seq) {
        if (std::find(b_seq.begin(), b_seq.end(), seq) != b_seq.end()) drop_batch();
    }
    void drop_batch() {
        runs_known = false;
        b_seq.clear();
        b_before.clear();
        b_fresh.clear();
    }
    void clear() {
        refs.assign(desc.n_pages, 0);
        free_w.assign((desc.n_pages + 63) / 64, ~0ull);
        if (desc.n_pages & 63) free_w.back() = (1ull << (desc.n_pages & 63)) - 1;
        first_free = 0;
        n_free = desc.n_pages;
        for (np::Seq& q : seqs) {
            q.pages.clear();
            q.tokens = q.stale_lo = q.stale_hi = 0;
        }
        seqs.resize(desc.max_seqs);
        stale.clear();
        drop_batch();
    }
    // Room that calls need after their checks: they change nothing unless all of it is there.
    void reserve() {
        stale.reserve(desc.max_seqs);  // each sequence once
        for (std::vector<int32_t>* v : {&b_seq, &b_before, &b_fresh}) v->reserve(np::kMaxBatch);
    }
    void reserve_pages(np::Seq& q, size_t n) const {
        if (n > q.pages.capacity()) q.pages.reserve(std::min<size_t>(std::max(n, 2 * q.pages.capacity()), desc.max_pages));
    }
    np::KvView view() const {
        np::KvView v;
        v.codes = static_cast<uint8_t*>(desc.codes);
        v.exps = desc.exps;
        v.table = table;
        v.page_bytes = page_bytes;
        v.layer_bytes = layer_bytes;
        v.n_pages = desc.n_pages;
        v.max_pages = desc.max_pages;
        v.page_shift = page_shift;
        v.n_heads = desc.n_heads;
        v.n_kv = desc.n_kv_heads;
        v.hd = desc.head_dim;
        v.slabs = slabs;
        return v;
    }
    ~np_kv() {
        if (table) (void)hipFree(table);
        if (part) (void)hipFree(part);
        if (arrived) (void)hipFree(arrived);
    }
};

namespace np {

// What every call that may enqueue checks first.
inline np_status check_kv(const np_kv* kv) {
    if (!kv) return fail(NP_EINVAL, "kv must not be NULL");
    if (kv->broken) return fail(NP_ESTATE, "an earlier call failed in the middle: call np_kv_reset");
    return NP_OK;
}

// Makes the cache's device current, if it has one: after the checks of a call, before it changes anything.
inline np_status make_current(const np_kv* kv, std::optional<DeviceGuard>& g) {
    if (kv->host_only()) return NP_OK;
    g.emplace(kv->desc.device);
    return g->ok ? NP_OK : fail(NP_EHIP, "hipSetDevice(%d) failed", kv->desc.device);
}

inline int elem_bytes(int32_t dtype) { return dtype == NP_F32 ? 4 : 2; }

inline np_status check_layer_io(const np_kv* kv, int32_t layer, int32_t dtype) {
    const np_status st = check_kv(kv);
    if (st != NP_OK) return st;
    if (layer < 0 || layer >= kv->desc.n_layers)
        return fail(NP_EINVAL, "layer %d out of range [0, %d)", layer, kv->desc.n_layers);
    if (dtype != NP_F32 && dtype != NP_BF16 && dtype != NP_F16) return fail(NP_EINVAL, "unknown dtype %d", dtype);
    if (kv->b_seq.empty()) return fail(NP_ESTATE, "no current tokens: call np_kv_extend first");
    return NP_OK;
}

inline np_status check_rows(const np_kv* kv, const void* p, int64_t row, int64_t head, int32_t dtype, const char* what) {
    if (!p || !aligned16(p)) return fail(NP_EINVAL, "%s must be a 16-byte aligned device pointer", what);
    const int64_t unit = 16 / elem_bytes(dtype);
    if (row < 0 || head < 0 || row % unit || head % unit || row > (int64_t)1 << 40 || head > (int64_t)1 << 40)
        return fail(NP_EINVAL, "%s: strides (%lld, %lld) must be multiples of 16 bytes, not negative", what,
                    (long long)row, (long long)head);
    return NP_OK;
}

// The checks of an attention call. S: the strides, given or contiguous; *rows: the current tokens.
inline np_status check_attend(const np_kv* kv, int32_t layer, const void* q, const void* out, const float* lse, int32_t dtype, const int64_t* strides,
                              float scale, int32_t window, int32_t sinks, int64_t* S, int64_t* n_rows) {
    np_status st = check_layer_io(kv, layer, dtype);
    if (st != NP_OK) return st;
    const np_kv_desc& D = kv->desc;
    if (!(std::isfinite(scale) && scale > 0.0f)) return fail(NP_EINVAL, "scale=%g must be positive and finite", scale);
    if (window < 0 || sinks < 0) return fail(NP_EINVAL, "window=%d and sinks=%d must not be negative", window, sinks);
    int64_t rows = 0;
    for (int32_t f : kv->b_fresh) rows += f;
    *n_rows = rows;
    const int64_t plain[4] = {(int64_t)D.n_heads * D.head_dim, D.head_dim, (int64_t)D.n_heads * D.head_dim, D.head_dim};
    for (int i = 0; i < 4; ++i) S[i] = strides ? strides[i] : plain[i];
    if ((st = check_rows(kv, q, S[0], S[1], dtype, "q")) != NP_OK) return st;
    if ((st = check_rows(kv, out, S[2], S[3], dtype, "out")) != NP_OK) return st;
    if (!((S[3] >= D.head_dim || D.n_heads == 1) && (S[2] >= (D.n_heads - 1) * S[3] + D.head_dim || rows <= 1)) &&
        !((S[2] >= D.head_dim || rows <= 1) && (S[3] >= (rows - 1) * S[2] + D.head_dim || D.n_heads == 1)))
        return fail(NP_EINVAL, "out: strides (%lld, %lld) make rows or heads overlap", (long long)S[2], (long long)S[3]);
    if (lse && ((uintptr_t)lse & 3u)) return fail(NP_EINVAL, "lse must be 4-byte aligned");
    if (kv->host_only()) return fail(NP_ESTATE, "a bookkeeping-only cache holds no tokens");
    if ((st = check_io_ptr(q, D.device, "q", "cache")) != NP_OK) return st;
    if ((st = check_io_ptr(out, D.device, "out", "cache")) != NP_OK) return st;
    if (lse && (st = check_io_ptr(lse, D.device, "lse", "cache")) != NP_OK) return st;
    return NP_OK;
}

// The current batch; items(i) gives the work items of its i-th sequence.
template <typename Batch, typename F>
void fill_batch(const np_kv* kv, Batch& b, F items) {
    b.n = (int32_t)kv->b_seq.size();
    int32_t row = 0, item = 0;
    for (int i = 0; i < b.n; ++i) {
        b.seq[i] = kv->b_seq[i];
        b.before[i] = kv->b_before[i];
        b.fresh[i] = kv->b_fresh[i];
        b.row0[i] = row;
        b.item0[i] = item;
        row += b.fresh[i];
        item += items(i);
    }
    b.item0[b.n] = item;
}

// No C++ exception leaves a C entry: the only ones here are failed host allocations.
template <typename F>
np_status guarded(F f) {
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return fail(NP_ENOMEM, "host allocation failed");
    } catch (...) {
        return fail(NP_EINVAL, "unexpected host error");
    }
}

}  // namespace np
