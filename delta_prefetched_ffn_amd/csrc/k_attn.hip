// Attention over the 8-bit key/value cache for gfx950 (format and semantics: include/np.h).
//
// For a query row at position i of a sequence and one of its heads, over the visible tokens j
// (j <= i, held, and inside the window or among the first tokens):
//     s_j = scale * q . k_j,   out = sum_j exp(s_j) v_j / sum_j exp(s_j),   lse = ln sum_j exp(s_j)
// with k_j = 2^ek * code, v_j = 2^ev * code of the token's block. One pass over the tokens with the
// running maximum m and sum l (base 2: s * log2(e) is folded into one factor per block).
//
// Everything stays in registers. The matrix products are transposed, S^T = K Q^T and
// O^T = V^T P^T, 16 rows (query token, head of the group) wide. The cache's tile order makes each
// lane's 16-byte chunk of a K tile its operand for two 16x16x32 products (codes become 16-bit
// floats exactly), and the S^T it receives (four tokens of one row) is, rounded to fp16, the
// operand of the second product: two groups of 16 tokens fill its 32 k-slots, four per lane and
// group, and the V tile's dword i of the lane's chunk holds exactly those four tokens of value
// 4 r + i. So neither P nor V crosses lanes, and a lane's results are 16 consecutive values.
#include <algorithm>
#include <atomic>

#include "attn_device.hpp"
#include "prefix_internal.hpp"

namespace np {
namespace {

constexpr int kRows = kRowTile;      // query rows of a tile
constexpr int kPiece = kPieceTokens;  // tokens of one step
// The tokens a row tile reads, as 32-token pieces: the first tokens' pieces, then those of
// [first, end).
struct Pieces {
    int n_sink, first, total;
    __device__ int operator[](int u) const { return u < n_sink ? u : first + (u - n_sink); }
};
__device__ inline Pieces pieces_of(int pos_lo, int pos_hi, int window, int sinks) {
    const int lo = window ? max(0, pos_lo - window + 1) : 0;
    Pieces p;
    p.n_sink = (min(sinks, lo) + kPiece - 1) / kPiece;
    p.first = max(p.n_sink, lo / kPiece);
    p.total = p.n_sink + pos_hi / kPiece + 1 - p.first;
    return p;
}

// Whether any row at positions pos_lo .. pos_hi sees any of the 16 tokens from t on. A group that none
// sees is treated as one that is not held: its values' scale must not decide what the others keep.
__device__ inline bool group_seen(const AttnArgs& a, int t, int pos_lo, int pos_hi) {
    return t <= pos_hi && (!a.window || pos_lo - (t + 15) < a.window || t < a.sinks);
}

// Four values of a finished row (query token and head of the group: r), and its lse.
template <typename T>
__device__ inline void store_row(const AttnArgs& a, int row0, int group, int h, int r, int d, f32x4 x, float ll, float mm) {
    const bool none = mm == -__builtin_inff() && ll == 0.0f;  // no visible token: 0
    const int t = r / group, head = h * group + r - t * group;
    T* const out = static_cast<T*>(a.out) + (int64_t)(row0 + t) * a.o_row + (int64_t)head * a.o_head + d;
    const float inv = none ? 0.0f : 1.0f / ll;
    T y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = (T)(x[j] * inv);
    __builtin_memcpy(__builtin_assume_aligned(out, 4 * sizeof(T)), y, sizeof y);
    if (a.lse && d == 0)
        a.lse[(int64_t)(row0 + t) * a.kv.n_heads + head] =
            none ? -__builtin_inff() : ll == 0.0f ? __builtin_nanf("") : (mm + __builtin_amdgcn_logf(ll)) * 0.69314718055994531f;
}

// Partial results pass between dies: stores and loads that bypass the die's own cache.
__device__ inline void put2(float* p, float x, float y) {
    const uint64_t w = (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x);
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p), w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline f32x2 get2(const float* p) {
    const uint64_t w = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return f32x2{__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}

// Few rows: one workgroup of W waves per (row tile, split of the key axis, kv head). Its waves take
// every W-th piece of the split and are joined through LDS; the workgroup that finishes a row tile
// last joins the splits, in their order (so the result does not depend on which one that is).
//
// Bound by the cache's bytes (4 * group products per byte). A wave asks for a piece's K and V (8 KiB
// at head_dim 128) a step ahead; page numbers and exponents of its next 32 pieces are fetched by its
// lanes in two loads, so a piece's address needs no memory round trip of its own. Measured where 256
// workgroups of 8 waves have 2, 4 and 63 pieces a wave (32 heads x 4 Ki tokens; 8 x 8 heads x 4 Ki; 24 x 8 heads x 4 .. 32 Ki): 4
// waves 15.2, 18.7 and 196 us, 8 waves 13.5, 18.5 and 192 us, 16 waves 15.7, 20.3 and 210 us.
template <typename T, int NS, int W>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(W / 4))) void k_attn_rows(AttnArgs a) {
    typedef AttnKind<T> Kd;
    typedef typename Kd::Q Q;
    typedef typename Kd::P P;
    typedef typename Vec8<Q>::t Q8;
    typedef typename Vec8<P>::t P8;
    const KvView& kv = a.kv;
    const int b = find_item(a.b, blockIdx.x), h = blockIdx.y;
    const int splits = a.b.splits[b], item = (int)blockIdx.x - a.b.item0[b], rt = item / splits, sp = item - rt * splits;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int group = kv.n_heads / kv.n_kv, rows = a.b.fresh[b] * group, r0 = rt * kRows;
    const int row = r0 + col;  // (query token, head of the group)
    const bool real = row < rows;
    const int tq = row / group, head = h * group + row - tq * group;
    const int before = a.b.before[b], pos = before + tq;
    const int pos_lo = before + r0 / group, pos_hi = before + min(r0 + kRows - 1, rows - 1) / group;
    const Pieces pc = pieces_of(pos_lo, pos_hi, a.window, a.sinks);
    const int share = pc.total / splits, more = pc.total - share * splits;
    const int u0 = sp * share + min(sp, more), u1 = u0 + share + (sp < more ? 1 : 0);

    const uint8_t* const codes = kv.codes + a.layer * kv.layer_bytes;
    const int8_t* const exps = kv.exps + (int64_t)a.layer * kv.n_pages * kv.n_kv * 2;
    const int side_bytes = (1 << kv.page_shift) * kv.slabs * kTileDims;
    const int seq = a.b.seq[b];

    // The wave's pieces are u0 + wave + n * W, n < count. Lane i: page and exponents of group i % 2 of
    // piece (n & ~31) + i / 2.
    const int count = u1 - u0 > wave ? (u1 - u0 - wave + W - 1) / W : 0;
    const auto token_of = [&](int n) { return pc[u0 + wave + n * W] * kPiece; };
    int ahead_page = -1, ahead_exps = 0;
    const auto fetch_pages = [&](int n0) {
        const int n = n0 + (lane >> 1), t = n < count ? token_of(n) + 16 * (lane & 1) : pos_hi + 1;
        ahead_page = group_seen(a, t, pos_lo, pos_hi) ? page_of(kv, seq, t >> kv.page_shift) : -1;
    };
    const auto fetch_exps = [&] {
        ahead_exps = *reinterpret_cast<const uint16_t*>(exps + ((int64_t)max(ahead_page, 0) * kv.n_kv + h) * 2);
    };
    // The q tile goes through LDS, one operand (c, f) per wave: all waves share it, and 16 waves at
    // 128 registers have none left for it. Its trip runs beside the first page numbers'.
    extern __shared__ __attribute__((aligned(128))) float s_mem[];
    Q8* const s_q = reinterpret_cast<Q8*>(s_mem);  // [NS][2][kQ][64 lanes]
    fetch_pages(0);
    for (int cf = wave; cf < 2 * NS; cf += W) {
        const int d = (cf >> 1) * 64 + quad * 16 + (cf & 1) * 8;
        const T* const qrow = static_cast<const T*>(a.q) + (int64_t)(a.b.row0[b] + tq) * a.q_row + (int64_t)head * a.q_head + d;
        u32x4 raw[sizeof(T) / 2];
#pragma unroll
        for (int w = 0; w < (int)sizeof(T) / 2; ++w) {
            raw[w] = u32x4{0, 0, 0, 0};
            if (real && d < kv.hd) raw[w] = reinterpret_cast<const u32x4*>(qrow)[w];
        }
        if constexpr (sizeof(T) == 2) {
            s_q[cf * 64 + lane] = __builtin_bit_cast(Q8, raw[0]);
        } else {
            float x[8];
            __builtin_memcpy(x, raw, sizeof x);
            Q8 t[Kd::kQ];
            split<Q, Kd::kQ>(t, x);
#pragma unroll
            for (int n = 0; n < Kd::kQ; ++n) s_q[(cf * Kd::kQ + n) * 64 + lane] = t[n];
        }
    }
    __syncthreads();

    f32x4 o[NS][4];
#pragma unroll
    for (int c = 0; c < NS; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[c][i] = f32x4{0, 0, 0, 0};
    float m = -__builtin_inff(), l = 0.0f;  // l: this lane's tokens only, joined at the end
    bool seen = false;
    int unit = kNoUnit, top = kNoUnit;  // o is in units of 2^unit

    // K of the next piece is asked for once this one's products have read K, V once they have read V:
    // a wave always has loads in flight and holds one piece only. The last piece's "next" loads read
    // one line of the pool's start, so that their number is the same in every turn (the wait for K or
    // V counts the loads behind it).
    u32x4 k[2][NS], v[2][NS];
    const uint8_t* at[2];  // of the piece whose K was asked for last
    int lane16 = lane * 16;
    const auto locate = [&](int n) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            // A group that is not held (or lies past the last position) reads page 0: its tokens are
            // hidden below like any other hidden token.
            const int page = max(0, __builtin_amdgcn_readlane(ahead_page, (n & 31) * 2 + g)), t = token_of(n) + 16 * g;
            at[g] = codes + page * kv.page_bytes + (int64_t)h * 2 * side_bytes +
                    (int64_t)((t & ((1 << kv.page_shift) - 1)) >> 4) * (kv.slabs * kTileBytes);
        }
    };
    const auto load_k = [&] {
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int c = 0; c < NS; ++c) k[g][c] = *reinterpret_cast<const u32x4*>(at[g] + c * kTileBytes + lane16);
    };
    const auto load_v = [&] {
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int c = 0; c < NS; ++c) v[g][c] = *reinterpret_cast<const u32x4*>(at[g] + side_bytes + c * kTileBytes + lane16);
    };
    fetch_exps();
    locate(0);
    if (!count) lane16 = 0;
    load_k();
    load_v();
    for (int n = 0; n < count; ++n) {
        const int tok = token_of(n);
        bool held[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) held[g] = __builtin_amdgcn_readlane(ahead_page, (n & 31) * 2 + g) >= 0;

        f32x4 acc[2];  // raw scores of tokens tok + 16 g + 4 quad + j
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            acc[g] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < NS; ++c)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const Q8 kk = widen<Q>(k[g][c][2 * f], k[g][c][2 * f + 1], 1.0f, 1.0f);
#pragma unroll
                    for (int t = 0; t < Kd::kQ; ++t) acc[g] = mfma(kk, s_q[((c * 2 + f) * Kd::kQ + t) * 64 + lane], acc[g]);
                }
        }
        __builtin_amdgcn_sched_barrier(0);
        float kf[2];
        int ev[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int e = __builtin_amdgcn_readlane(ahead_exps, (n & 31) * 2 + g);
            kf[g] = a.scale2 * pow2i(max(-126, (int)(int8_t)e));
            ev[g] = max(-126, (int)(int8_t)(e >> 8));
        }
        if (n + 1 < count) {
            if ((n & 31) == 31) {
                fetch_pages(n + 1);
                fetch_exps();
                asm volatile("" : "+v"(ahead_exps));  // waited for here, in this branch
            }
            locate(n + 1);
        } else {
            at[0] = at[1] = codes;
            lane16 = 0;
        }
        load_k();

        float s[8];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[4 * g + j] = acc[g][j] * kf[g];
        // Visibility: a piece that every row of the tile sees whole needs no comparisons.
        const bool whole = held[0] && held[1] && tok + kPiece - 1 <= pos_lo &&
                           (!a.window || tok > pos_hi - a.window || tok + kPiece <= a.sinks);
        uint32_t vis = 0xff;
        if (!whole) {
            vis = 0;
#pragma unroll
            for (int k8 = 0; k8 < 8; ++k8) {
                const int t = tok + 16 * (k8 >> 2) + 4 * quad + (k8 & 3);
                const bool ok = t <= pos && held[k8 >> 2] && (!a.window || pos - t < a.window || t < a.sinks);
                vis |= ok ? 1u << k8 : 0u;
                if (!ok) s[k8] = -__builtin_inff();
            }
        }
        seen |= vis != 0;
        float mx = s[0];
#pragma unroll
        for (int k8 = 1; k8 < 8; ++k8) mx = fmaxf(mx, s[k8]);
        if (__any(mx > m + kLazy)) {
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float m1 = fmaxf(m, mx);
            const float f = m1 == m ? 1.0f : __builtin_amdgcn_exp2f(m - m1);
            m = m1;
            l *= f;
#pragma unroll
            for (int c = 0; c < NS; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[c][i] *= f;
        }
        const float m0 = (m == -__builtin_inff() ? 0.0f : m) - Kd::kLift;  // 0: a row that has seen nothing finite
        float p[8];
#pragma unroll
        for (int k8 = 0; k8 < 8; ++k8) {
            p[k8] = __builtin_amdgcn_exp2f(s[k8] - m0);
            if (!(vis >> k8 & 1)) p[k8] = 0.0f;
            l += p[k8];
        }

        // O += V^T P^T. Both groups at once, or one at a time where their V scales lie too far apart for
        // one unit (the other group's codes are then out of the product: they would overflow).
        const auto fit_unit = [&](int ea, int eb) {
            const int lo_e = min(ea, eb), hi_e = max(ea, eb);
            top = max(top, hi_e);
            const int to = max(min(hi_e, lo_e + kFar), top - kDrop);
            if (to != unit && (hi_e > unit + kNear || lo_e < unit - kFar)) {
                const float f = pow2i(max(-126, unit - to));
#pragma unroll
                for (int c = 0; c < NS; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[c][i] *= f;
                unit = to;
            }
        };
        // Exponents of groups that are not held are page 0's: they must not move the unit.
        const int e0 = held[0] ? ev[0] : held[1] ? ev[1] : unit, e1 = held[1] ? ev[1] : e0;
        const bool near = e0 - e1 <= kNear + kFar && e1 - e0 <= kNear + kFar;
        // NaN codes of tokens that a row does not see must not reach it: 0 * NaN is NaN. Tokens that no row
        // of the tile sees (often bytes never written) are cleared here; the path below keeps real NaN
        // values from the rows that do not see them.
        bool clean = true;
        if (!whole) {
            uint32_t bad = 0;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint32_t some = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = tok + 16 * g + 4 * quad + j;
                    if (held[g] && t <= pos_hi && (!a.window || pos_lo - t < a.window || t < a.sinks)) some |= 0xffu << (8 * j);
                }
#pragma unroll
                for (int c = 0; c < NS; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[g][c][i] &= some;
                        bad |= nan_bytes(v[g][c][i]);
                    }
            }
            clean = !__any(bad != 0);
        }
        if (clean && near) {
            fit_unit(e0, e1);
            const float f0 = pow2i(max(-126, e0 - unit)), f1 = pow2i(max(-126, e1 - unit));
            P8 pv[Kd::kP];
            split<P, Kd::kP>(pv, p);
#pragma unroll
            for (int c = 0; c < NS; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const P8 vv = widen<P>(v[0][c][i], v[1][c][i], f0, f1);
#pragma unroll
                    for (int t = 0; t < Kd::kP; ++t) o[c][i] = mfma(vv, pv[t], o[c][i]);
                }
        } else {
        // Row by row, each with the codes of the tokens it sees and, of two far scales, one at a time.
        for (int turn = 0; turn < (near ? kRows : 2 * kRows); ++turn) {
            const int r = turn & (kRows - 1), pass = turn / kRows;
            const int ea = near ? e0 : pass ? e1 : e0, eb = near ? e1 : ea;
            fit_unit(ea, eb);
            const float f0 = pow2i(max(-126, ea - unit)), f1 = pow2i(max(-126, eb - unit));
            const uint32_t vr = __shfl(vis, quad * 16 + r);
            uint32_t in[2] = {0, 0};
#pragma unroll
            for (int k8 = 0; k8 < 8; ++k8)
                if ((vr >> k8 & 1) && (near || (k8 >> 2) == pass)) in[k8 >> 2] |= 0xffu << (8 * (k8 & 3));
            P8 pv[Kd::kP];
            split<P, Kd::kP>(pv, p);
#pragma unroll
            for (int c = 0; c < NS; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const P8 vv = widen<P>(v[0][c][i] & in[0], v[1][c][i] & in[1], f0, f1);
                    f32x4 x = o[c][i];
#pragma unroll
                    for (int t = 0; t < Kd::kP; ++t) x = mfma(vv, pv[t], x);
                    if (col == r) o[c][i] = x;
                    __builtin_amdgcn_sched_barrier(0);  // this path must not cost registers
                }
        }
        }
        load_v();
    }

    // Join the waves: rows' maximum, sum and O in true units.
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    l *= 1.0f / (1 << Kd::kLift);
    seen = (__ballot(seen) >> col & 0x0001000100010001ull) != 0;
    // Every score this wave saw is -inf. Beside finite scores they weigh 0; if the whole row's are, it is 0 / 0. The
    // lowest finite maximum joins as just that.
    if (seen && m == -__builtin_inff()) m = -__FLT_MAX__;
    constexpr int D = NS * 64, DS = D + 4;
    __syncthreads();  // the q tile is done with
    const int cap = a.row_cap;
    float* const s_m = s_mem;  // [W][cap]
    float* const s_l = s_m + W * cap;
    float* const s_o = s_l + W * cap;  // [W][cap][DS]
    const int tile_rows = min(kRows, rows - r0);
    const float back = __builtin_amdgcn_ldexpf(1.0f, unit - Kd::kLift);
    if (col < tile_rows) {
        float* const dst = s_o + (wave * cap + col) * DS + quad * 16;
#pragma unroll
        for (int c = 0; c < NS; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<f32x4*>(dst + c * 64 + 4 * j) = f32x4{o[c][0][j], o[c][1][j], o[c][2][j], o[c][3][j]} * back;
        if (quad == 0) {
            s_m[wave * cap + col] = m;
            s_l[wave * cap + col] = l;
        }
    }
    __syncthreads();
    const int D4 = kv.hd / 4, n_out = tile_rows * D4;
    const int64_t first = ((int64_t)(a.b.part0[b] + rt * splits) * kv.n_kv + h), step = kv.n_kv;
    const int PS = cap * (D + 2);
    for (int k = threadIdx.x; k < n_out; k += 64 * W) {
        const int r = k / D4, d = (k - r * D4) * 4;
        float mm = s_m[r], ll = 0.0f;
#pragma unroll 4
        for (int w = 1; w < W; ++w) mm = fmaxf(mm, s_m[w * cap + r]);
        f32x4 x = {0, 0, 0, 0};
#pragma unroll 4
        for (int w = 0; w < W; ++w) join(x, ll, mm, s_m[w * cap + r], s_l[w * cap + r], *reinterpret_cast<const f32x4*>(s_o + (w * cap + r) * DS + d));
        if (splits == 1) {
            store_row<T>(a, a.b.row0[b], group, h, r0 + r, d, x, ll, mm);
        } else {
            // Past the caches of this die, to where the joining workgroup reads.
            float* const part = a.part + (first + sp * step) * PS + r * (D + 2);
            put2(part + 2 + d, x[0], x[1]);
            put2(part + 4 + d, x[2], x[3]);
            if (d == 0) put2(part, mm, ll);
        }
    }
    if (splits == 1) return;
    // Each wave's stores are done (acknowledged where every die sees them) before the count rises.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    uint32_t* const s_last = reinterpret_cast<uint32_t*>(s_mem);
    if (threadIdx.x == 0) s_last[0] = atomicInc(a.arrived + first, (uint32_t)splits - 1);  // back to 0 with the last
    __syncthreads();
    if (s_last[0] != (uint32_t)splits - 1) return;
    for (int k = threadIdx.x; k < n_out; k += 64 * W) {
        const int r = k / D4, d = (k - r * D4) * 4;
        const float* const p = a.part + first * PS + r * (D + 2);
        float mm = -__builtin_inff(), ll = 0.0f;
        f32x4 x = {0, 0, 0, 0};
        constexpr int U = 4;  // splits in flight
        for (int s0 = 0; s0 < splits; s0 += U) {
            f32x2 ml[U], xa[U], xb[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float* const q = p + min(s0 + i, splits - 1) * step * PS;
                ml[i] = get2(q);
                xa[i] = get2(q + 2 + d);
                xb[i] = get2(q + 4 + d);
            }
            float m1 = mm;
#pragma unroll
            for (int i = 0; i < U; ++i) m1 = fmaxf(m1, ml[i][0]);
            if (m1 != mm) {
                const float f = __builtin_amdgcn_exp2f(mm - m1);
                x *= f;
                ll *= f;
                mm = m1;
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (s0 + i < splits) join(x, ll, mm, ml[i][0], ml[i][1], f32x4{xa[i][0], xa[i][1], xb[i][0], xb[i][1]});
        }
        store_row<T>(a, a.b.row0[b], group, h, r0 + r, d, x, ll, mm);
    }
}

// Waves of a workgroup for many rows: 8, two to a SIMD at 256 registers, where q, O and the scores fit; 4
// at 512 registers for heads above 192 values, one to a SIMD, so without the half-step distance. At 192
// values they do not quite fit: 38 (bf16) or 46 (fp16) registers are spilled, to 156 bytes of scratch a
// lane. A causal prompt of 4 Ki tokens x 32 heads takes 136 us at 64 values, 306 us at 192 and 652 us at
// 256, where the products at a large library product's rate would take 51, 152 and 203.
template <int NS>
constexpr int kTileWaves = NS <= 3 ? 8 : 4;

// x, computed before what follows in the program: the compiler moves arithmetic across barriers.
template <typename V>
__device__ inline V settled(V x) {
    u32x4 w = __builtin_bit_cast(u32x4, x);
    asm volatile("" : "+v"(w));
    return __builtin_bit_cast(V, w);
}

// Many rows: one workgroup of W waves per (32 W rows, kv head), 32 rows a wave, 64 tokens a step.
//
// Per 64 tokens a wave has 32 products of 32x32x16 (33 clocks each) and 32 exponentials a lane. Codes
// are widened to 16 bits once per workgroup, by the wave that moved them into LDS (every wave reads
// them all, 1 KiB of consecutive operands at a time), with V's scale folded into that conversion; the
// products are transposed as above, so P needs no trip through LDS. The two waves of a SIMD are half a
// step apart: one's products run beside the other's softmax and moves. Neighbouring workgroups are of
// different kv heads, so a head's row tiles run on one die (8 divides most head counts), whose cache
// then holds its K and V; the longest rows come first.
//
// Measured at head_dim 128: a causal prompt of 4 Ki tokens x 32 heads 165 us, 833 TFLOP/s (a large
// library product reaches 1,354); 8,191 tokens x 32 over 8 heads with a window of 4 Ki 461 us, 895
// TFLOP/s. A step takes about 4,900 clocks where its products need 2,112: a wave alone reads LDS at 33
// bytes a clock, one operand per product's time (62 clocks for both; 33 with two waves), and the vector
// work (masks and maxima 600, exponentials 610, widening 800 for K and 1,360 for V) of two waves
// is longer than their products. Without the half-step distance 175 us; with codes moved by all waves at
// the end of a step 187 us.
//
// Operand slots: S^T lane (half, row) holds tokens 8 (i / 4) + 4 half + i % 4, i < 16, of a 32-token
// block; so slot j of the second product is token 8 (j / 4) + 4 half + j % 4 of a 16-token group, i.e.
// V quads half and 2 + half. Row rho of V^T tile (slab, vt) is value 64 slab + 4 (rho % 16) + 2 vt +
// rho / 16: then the lanes that widen V write without bank conflicts, and a lane ends with runs of 16
// consecutive values of its row.
template <typename T, int NS, int W>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(W / 4))) void k_attn_tile(AttnArgs a) {
    typedef AttnKind<T> Kd;
    typedef typename Kd::Q Q;
    typedef typename Kd::P P;
    typedef typename Vec8<Q>::t Q8;
    typedef typename Vec8<P>::t P8;
    constexpr int KS = NS * 4;               // 16-value steps of a head
    constexpr int kSide = 64 * NS * 64;      // values of a step's K (or V)
    constexpr bool kShift = W == 8;          // two waves to a SIMD, in opposite phases
    constexpr int kUnits = 8 * NS / W;       // 1 KiB code tiles a wave moves per step
    const KvView& kv = a.kv;
    const int item_all = blockIdx.x / kv.n_kv, h = blockIdx.x - item_all * kv.n_kv;
    const int b = find_item(a.b, item_all);
    const int rt = a.b.item0[b + 1] - 1 - item_all;  // the last rows first
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
    const int group = kv.n_heads / kv.n_kv, rows = a.b.fresh[b] * group, r0 = rt * 32 * W, w0 = r0 + 32 * wave;
    const int row = w0 + col;
    const bool real = row < rows;
    const int tq = row / group, head = h * group + row - tq * group;
    const int before = a.b.before[b], pos = before + tq;
    const int wg_lo = before + r0 / group, wg_hi = before + min(r0 + 32 * W - 1, rows - 1) / group;
    const int pos_lo = before + min(w0, rows - 1) / group, pos_hi = before + min(w0 + 31, rows - 1) / group;
    const int seq = a.b.seq[b];
    const float scale2 = a.scale2;
    const uint8_t* const codes = kv.codes + a.layer * kv.layer_bytes;
    const int8_t* const exps = kv.exps + (int64_t)a.layer * kv.n_pages * kv.n_kv * 2;
    const int side_bytes = (1 << kv.page_shift) * kv.slabs * kTileDims;

    // Steps of 64 tokens: the first tokens' steps, then those of the window.
    const int lo = a.window ? max(0, wg_lo - a.window + 1) : 0;
    const int n_sink = (min(a.sinks, lo) + 63) / 64, first = max(n_sink, lo / 64), steps = n_sink + wg_hi / 64 + 1 - first;
    const auto token_of = [&](int n) { return (n < n_sink ? n : first + n - n_sink) * 64; };

    // Lane i: group i % 4 of step (n & ~15) + i / 4: its K codes' address (page 0 where it is not held or
    // past the last position), exponents, and whether it is held.
    uint64_t ahead_at = 0;
    int ahead_exps = 0;
    bool ahead_held = false;
    const auto fetch = [&](int n0) __attribute__((always_inline)) {
        const int own = here(lane), n = n0 + (own >> 2), t = n < steps ? token_of(n) + 16 * (own & 3) : wg_hi + 1;
        const int page = group_seen(a, t, wg_lo, wg_hi) ? page_of(kv, seq, t >> kv.page_shift) : -1;
        ahead_held = page >= 0;
        ahead_exps = *reinterpret_cast<const uint16_t*>(exps + ((int64_t)max(page, 0) * kv.n_kv + h) * 2);
        ahead_at = reinterpret_cast<uint64_t>(codes + max(page, 0) * kv.page_bytes + (int64_t)2 * h * side_bytes +
                                              (int64_t)((t & ((1 << kv.page_shift) - 1)) >> 4) * (kv.slabs * kTileBytes));
        asm volatile("" : "+v"(ahead_exps));  // waited for here
        // A group that is not held has page 0's codes, whose exponent the unit knows nothing of. Its weights are 0, but
        // codes that overflow would be infinities, and 0 times those NaN: the lowest exponent keeps them small.
        if (page < 0) ahead_exps = 0x8000;
    };
    fetch(0);

    Q8 q[KS][Kd::kQ];
    {
        const T* const qrow = static_cast<const T*>(a.q) + (int64_t)(a.b.row0[b] + tq) * a.q_row + (int64_t)head * a.q_head;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int d = k * 16 + half * 8;
            float x[8] = {};
            if (real && d < kv.hd) load_row<8>(x, qrow + d);
            split<Q, Kd::kQ>(q[k], x);
        }
    }

    extern __shared__ __attribute__((aligned(128))) float s_mem[];
    Q* const s_k = reinterpret_cast<Q*>(s_mem);                // [2][2 blocks][KS][2 halves][32 tokens][8]
    P* const s_v = reinterpret_cast<P*>(s_mem) + 2 * kSide;    // [2][4 groups][2 NS][2 halves][32 rho][8]
    // Per step: the groups' K factors, a bit per token of held groups, the groups' V units; whether a V
    // code is NaN and, per value, the tokens where it is.
    __shared__ __attribute__((aligned(16))) float s_kf[2][4];
    __shared__ uint64_t s_held[2];
    __shared__ __attribute__((aligned(16))) int s_unit[2][4];
    __shared__ int s_has_nan[4];
    __shared__ unsigned long long s_nan[4][NS * 64];
    __shared__ uint32_t s_bad[32 * W][2 * NS];  // per row, a bit per value: it is NaN

    // What this wave moves in a step: kUnits of the code tiles [side][group][slab]. In opposite phases
    // the first waves move K, the others V.
    const bool second = kShift && wave >= W / 2;
    const bool moves_k = !kShift || !second, moves_v = !kShift || second;
    const auto tile_at = [&](int j, int& side, int& g, int& c) __attribute__((always_inline)) {
        const int tile = kShift ? (second ? 4 * NS : 0) + (wave & 3) + 4 * j : wave + W * j;
        side = tile / (4 * NS);
        g = tile / NS & 3;
        c = tile % NS;
    };
    u32x4 part[kUnits];
    const auto ask = [&](int n) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            int side, g, c;
            tile_at(j, side, g, c);
            const int from = (n & 15) * 4 + g;
            const uint64_t at = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(ahead_at >> 32), from) << 32 |
                                (uint32_t)__builtin_amdgcn_readlane((int)ahead_at, from);
            typedef const __attribute__((address_space(1))) u32x4 chunk;
            part[j] = reinterpret_cast<chunk*>(at + side * side_bytes + c * kTileBytes)[lane];
        }
    };
    int v_unit = 0, v_top = 0;
    bool begun = false, nan_met = false;  // nan_met: some step so far had a NaN
    const auto put = [&](int n) __attribute__((always_inline)) {
        const int buf = n & 1, from = (n & 15) * 4, my_ev = max(-126, (int)(int8_t)(ahead_exps >> 8));
        const uint32_t holds = (uint32_t)(__ballot(ahead_held) >> from) & 15;
        if (wave == 0 && lane >> 2 == (n & 15)) {
            // K's factor is never 0: a hidden score is -inf, and stays it times this.
            s_kf[buf][lane & 3] = fmaxf(scale2 * pow2i(max(-126, (int)(int8_t)ahead_exps)), 1.2e-38f);
            if ((lane & 3) == 0) s_held[buf] = (holds & 1 ? 0xffffull : 0) | (holds & 2 ? 0xffffull << 16 : 0) | (holds & 4 ? 0xffffull << 32 : 0) | (holds & 8 ? 0xffffull << 48 : 0);
        }
        if (moves_v) {
            // The V units of the step's groups, in order (every wave works out the same). Mostly all are near
            // the unit, and it stays.
            const bool fits = my_ev <= v_unit + kNear && my_ev >= v_unit - kFar;
            int un[4] = {v_unit, v_unit, v_unit, v_unit};
            if (!begun || ((uint32_t)(__ballot(ahead_held && !fits) >> from) & 15)) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int e = __builtin_amdgcn_readlane(my_ev, from + g);
                    if (holds >> g & 1) {
                        v_top = begun ? max(v_top, e) : e;
                        if (!begun || e > v_unit + kNear || e < v_unit - kFar) v_unit = max(e, v_top - kDrop);
                        begun = true;
                    }
                    un[g] = v_unit;
                }
            }
            if (wave == (kShift ? W / 2 : 0) && lane < 4) s_unit[buf][lane] = lane < 2 ? (lane ? un[1] : un[0]) : lane == 2 ? un[2] : un[3];
            // The notes of the step before the last are done with.
            if (nan_met) {
                for (int i = threadIdx.x & (W * 32 - 1); i < NS * 64; i += W * 32) s_nan[(n + 2) & 3][i] = 0;
            }
#pragma unroll
            for (int j = 0; j < kUnits; ++j) {
                int side, g, c;
                tile_at(j, side, g, c);
                if (side == 0) continue;
                const int e = __builtin_amdgcn_readlane(my_ev, from + g), u = g < 2 ? (g ? un[1] : un[0]) : g == 2 ? un[2] : un[3];
                const int quad = lane >> 4, r = lane & 15;
                uint32_t bad = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) bad |= nan_bytes(part[j][i]);
                if (__any(bad != 0)) {
                    // NaN codes must not reach rows that do not see their token (0 * NaN is NaN): they leave
                    // the product, and a note of them gives them back to the rows that do. Tokens that nobody
                    // sees (dropped, or past the last position: often bytes never written) leave no note.
                    const bool live = (holds >> g & 1) != 0;
                    const int own = here(lane), place = 16 * g + 4 * (own >> 4), t = token_of(n) + place;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t nb = nan_bytes(part[j][i]);
                        uint64_t at = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if ((nb >> (8 * k + 7) & 1) && live && t + k <= wg_hi) at |= 1ull << (place + k);
                        if (at) {
                            atomicOr(&s_nan[n & 3][64 * c + 4 * (own & 15) + i], (unsigned long long)at);
                            s_has_nan[n & 3] = 1;
                        }
                        part[j][i] &= ~((nb >> 7) * 255u);
                    }
                }
                const float f = pow2i(max(-126, min(127, e - u)));
                // value 4 r + i: tile vt = i / 2, rho = r + 16 (i % 2); half quad % 2, slots 4 (quad / 2) ..
                u32x2* const d = reinterpret_cast<u32x2*>(s_v + buf * kSide) + ((g * NS + c) * 2 * 64 + (quad & 1) * 32 + r) * 2 + (quad >> 1);
                const u32x4 xw = __builtin_bit_cast(u32x4, widen<P>(part[j][0], part[j][1], f, f));
                const u32x4 yw = __builtin_bit_cast(u32x4, widen<P>(part[j][2], part[j][3], f, f));
                d[0] = u32x2{xw[0], xw[1]};
                d[32] = u32x2{xw[2], xw[3]};
                d[128] = u32x2{yw[0], yw[1]};
                d[160] = u32x2{yw[2], yw[3]};
            }
        }
        if (moves_k) {
#pragma unroll
            for (int j = 0; j < kUnits; ++j) {
                int side, g, c;
                tile_at(j, side, g, c);
                if (side != 0) continue;
                Q8* const d = reinterpret_cast<Q8*>(s_k + buf * kSide) + ((g >> 1) * KS + c * 4 + (lane >> 4)) * 64 + (g & 1) * 16 + (lane & 15);
                d[0] = widen<Q>(part[j][0], part[j][1], 1.0f, 1.0f);
                d[32] = widen<Q>(part[j][2], part[j][3], 1.0f, 1.0f);
            }
        }
    };

    f32x16 o[2 * NS];
#pragma unroll
    for (int i = 0; i < 2 * NS; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f;  // l: this lane's tokens only
    bool seen = false;
    int unit = 0;

    for (int i = threadIdx.x; i < 4 * NS * 64; i += 64 * W) s_nan[0][i] = 0;
    for (int i = threadIdx.x; i < 64 * W * NS; i += 64 * W) s_bad[0][i] = 0;
    if (threadIdx.x < 4) s_has_nan[threadIdx.x] = 0;
    ask(0);
    __syncthreads();
    put(0);
    if (steps > 1) ask(1);
    // A wave's step n: between barriers the softmax of step n and the move of step n + 1, then the
    // products of K(n + 1) and of V(n). The two waves of a SIMD are half a step apart, so one has the matrix
    // unit while the other has the vector unit. The second half's V(n + 1) takes the buffer that
    // everybody's products of V(n - 1) are done with, the first half's K(n + 1) that of K(n - 1).
    P8 pv[4][Kd::kP];
    uint64_t vis = 0;
    f32x16 s[2];
    // The products of K(n) (S = 0 first) and of V(n - 1), interleaved: a sum's next product is issued
    // when the last one's result is there. Operands come from LDS a few products ahead.
    const auto products = [&](int n, bool first) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) s[t][j] = 0.0f;
        const Q8* const kt = reinterpret_cast<const Q8*>(s_k + (n & 1) * kSide) + lane;
        const P8* const vt = reinterpret_cast<const P8*>(s_v + (~n & 1) * kSide) + lane;
        constexpr int kMfma = 0x8, kDsRead = 0x100;  // classes of the scheduler
#pragma unroll
        for (int k = 0; k < 2 * KS; ++k) {  // 2 KS = 8 NS products of each kind
            const Q8 kk = kt[((k & 1) * KS + (k >> 1)) * 64];
#pragma unroll
            for (int x = 0; x < Kd::kQ; ++x) s[k & 1] = mfma(kk, q[k >> 1][x], s[k & 1]);
            if (first) continue;
            const P8 vv = vt[k * 64];
#pragma unroll
            for (int x = 0; x < Kd::kP; ++x) o[k % (2 * NS)] = mfma(vv, pv[k / (2 * NS)][x], o[k % (2 * NS)]);
        }
        constexpr int kAhead = 4;
        __builtin_amdgcn_sched_group_barrier(kDsRead, kAhead, 0);
#pragma unroll
        for (int i = 0; i < (first ? 2 : 4) * KS - kAhead; ++i) {
            __builtin_amdgcn_sched_group_barrier(kMfma, Kd::kQ, 0);  // kQ = kP
            __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(kMfma, kAhead * Kd::kQ, 0);
    };
    __syncthreads();
    if (second) __syncthreads();
    f32x4 kf = *reinterpret_cast<const f32x4*>(s_kf[0]);
    uint64_t held = s_held[0];
    products(0, true);
    for (int n = 0; n < steps; ++n) {
        const int buf = n & 1, tok = token_of(n);
        __syncthreads();
        // Read here, used behind the exponentials.
        const int has_nan_v = s_has_nan[n & 3];
        const u32x4 un_v = *reinterpret_cast<const u32x4*>(s_unit[buf]);
        const bool whole = held == ~0ull && tok + 63 <= pos_lo && (!a.window || tok > pos_hi - a.window || tok + 64 <= a.sinks);
        vis = ~0ull;  // of the row, a bit per token
        if (!whole) {
            const auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };
            vis = below(pos - tok + 1) & held;
            if (a.window) vis &= ~below(pos - a.window + 1 - tok) | below(a.sinks - tok);
            const uint64_t mine = vis >> (4 * half);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int bit = 8 * (i >> 2) + (i & 3);
                const int keep = (int)((uint32_t)(mine >> (bit & 32)) << (31 - (bit & 31))) >> 31;
                s[i >> 4][i & 15] = __uint_as_float((__float_as_uint(s[i >> 4][i & 15]) & keep) | (0xff800000u & ~keep));
            }
        }
        seen |= vis != 0;
        float mx = -__builtin_inff();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float x = s[g >> 1][8 * (g & 1)];
#pragma unroll
            for (int j = 1; j < 8; ++j) x = fmaxf(x, s[g >> 1][8 * (g & 1) + j]);
            mx = fmaxf(mx, x * kf[g]);
        }
        if (__any(mx > m + kLazy)) {
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float m1 = fmaxf(m, mx);
            const float f = m1 == m ? 1.0f : __builtin_amdgcn_exp2f(m - m1);
            m = m1;
            l *= f;
#pragma unroll
            for (int i = 0; i < 2 * NS; ++i) o[i] *= f;
        }
        const float m0 = (m == -__builtin_inff() ? 0.0f : m) - Kd::kLift;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[g >> 1][8 * (g & 1) + j], kf[g], -m0));
                l += p[j];
            }
            split<P, Kd::kP>(pv[g], p);
#pragma unroll
            for (int x = 0; x < Kd::kP; ++x) pv[g][x] = settled(pv[g][x]);  // in this phase, not behind the barrier
        }
        if (n + 1 < steps) {
            put(n + 1);
            if (n + 2 < steps) {
                if (((n + 2) & 15) == 0) fetch(n + 2);
                ask(n + 2);
            }
        }
        __syncthreads();
        int un[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) un[g] = __builtin_amdgcn_readfirstlane((int)un_v[g]);
        const bool has_nan = __builtin_amdgcn_readfirstlane(has_nan_v) != 0;
        nan_met |= has_nan;
        if (un[0] != unit || un[1] != unit || un[2] != unit || un[3] != unit) {
            // A change of unit. If not all groups share the new one, their products are made here, one
            // group after the other, and the weights below are zero.
            const bool one = un[0] == un[1] && un[0] == un[2] && un[0] == un[3];
            const P8* const vt = reinterpret_cast<const P8*>(s_v + buf * kSide) + lane;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float f = pow2i(max(-126, min(127, unit - un[g])));
                unit = un[g];
#pragma unroll
                for (int i = 0; i < 2 * NS; ++i) {
                    o[i] *= f;
                    if (!one) {
#pragma unroll
                        for (int x = 0; x < Kd::kP; ++x) o[i] = mfma(vt[(g * 2 * NS + i) * 64], pv[g][x], o[i]);
                    }
                    __builtin_amdgcn_sched_barrier(0);  // a rare path that must not cost registers
                }
#pragma unroll
                for (int x = 0; x < Kd::kP; ++x)
                    if (!one) pv[g][x] = __builtin_bit_cast(P8, u32x4{0, 0, 0, 0});
            }
        }
        // Behind the last step the scores are of no use (its K buffer holds an old step), but cost no branch.
        kf = *reinterpret_cast<const f32x4*>(s_kf[buf ^ 1]);  // of step n + 1
        held = s_held[buf ^ 1];
        products(n + 1, false);
        if (has_nan) {
            // Which values of this row meet a NaN: kept aside, for the end.
            const unsigned long long* const notes = s_nan[n & 3] + here(half) * 32 * NS;
#pragma unroll 1
            for (int w = 0; w < NS; ++w) {
                uint32_t word = 0;
#pragma unroll 1
                for (int d = 0; d < 32; ++d) word |= (notes[32 * w + d] & vis) ? 1u << d : 0u;
                s_bad[wave * 32 + col][half * NS + w] |= word;
            }
        }
    }
    if (kShift && !second) __syncthreads();

    l += __shfl_xor(l, 32);
    l *= 1.0f / (1 << Kd::kLift);
    seen = (__ballot(seen) >> col & 0x0000000100000001ull) != 0;
    if (!real) return;
    // Every visible score -inf: 0 / 0. No visible token: 0.
    const float inv = !seen ? 0.0f : m == -__builtin_inff() ? __builtin_nanf("") : 1.0f / l;
    const float back = __builtin_amdgcn_ldexpf(1.0f, unit - Kd::kLift);
    T* const out = static_cast<T*>(a.out) + (int64_t)(a.b.row0[b] + tq) * a.o_row + (int64_t)head * a.o_head;
#pragma unroll
    for (int c = 0; c < NS; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // eight values: run i / 2, its half i % 2
            const int d = 64 * c + 32 * (i >> 1) + 16 * half + 8 * (i & 1);
            if (d >= kv.hd) continue;
            const uint32_t bad = s_bad[wave * 32 + col][d >> 5] >> (d & 31);
            T y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // d + e = 64 c + 4 rho' + 2 vt + hi with rho' = 8 (i / 2) + 4 half + j, rho = rho' + 16 hi
                const int j = 2 * (i & 1) + (e >> 2), vt = e >> 1 & 1, hi = e & 1;
                const float x = seen ? o[2 * c + vt][4 * ((i >> 1) + 2 * hi) + j] * back * inv : 0.0f;
                y[e] = (T)(bad >> e & 1 ? __builtin_nanf("") : x);
            }
            __builtin_memcpy(__builtin_assume_aligned(out + d, 16), y, sizeof y);
        }
    if (a.lse && half == 0)
        a.lse[(int64_t)(a.b.row0[b] + tq) * kv.n_heads + head] =
            !seen ? -__builtin_inff() : m == -__builtin_inff() ? __builtin_nanf("") : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
}

// LDS of k_attn_rows per row of its tile (the join), and of k_attn_tile (two steps of K and V, 16 bits
// a value).
template <int NS>
constexpr size_t kRowLds = (size_t)kAttnWaves * (2 + NS * 64 + 4) * sizeof(float);
template <int NS>
constexpr int kTileLds = 4 * 64 * NS * 64 * 2;

template <typename T, int NS>
hipError_t tile_as(const AttnArgs& a, hipStream_t s) {
    constexpr int W = kTileWaves<NS>;
    k_attn_tile<T, NS, W><<<(unsigned)a.b.item0[a.b.n] * a.kv.n_kv, 64 * W, kTileLds<NS>, s>>>(a);
    return hipGetLastError();
}

template <typename T, int NS>
hipError_t rows_as(const AttnArgs& a, hipStream_t s) {
    constexpr int W = kAttnWaves;
    const dim3 grid(a.b.item0[a.b.n], a.kv.n_kv);
    const size_t lds = std::max(kRowLds<NS> * a.row_cap, sizeof(bf16x8) * 64 * 2 * NS * AttnKind<T>::kQ);
    k_attn_rows<T, NS, W><<<grid, 64 * W, lds, s>>>(a);
    return hipGetLastError();
}

template <typename T, int NS>
hipError_t tile_16(const AttnArgs& a, hipStream_t s) {
    if constexpr (sizeof(T) == 2) return tile_as<T, NS>(a, s);
    return hipErrorInvalidValue;  // attn_tile_rows() gives fp32 no tiles here
}

template <typename T>
hipError_t attn_as(const AttnArgs& a, hipStream_t s) {
    switch (a.kv.slabs) {
        case 1: return a.part ? rows_as<T, 1>(a, s) : tile_as<T, 1>(a, s);
        case 2: return a.part ? rows_as<T, 2>(a, s) : tile_16<T, 2>(a, s);
        case 3: return a.part ? rows_as<T, 3>(a, s) : tile_16<T, 3>(a, s);
        default: return a.part ? rows_as<T, 4>(a, s) : tile_16<T, 4>(a, s);
    }
}

template <typename T, int NS>
hipError_t prepare() {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_attn_rows<T, NS, kAttnWaves>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, (int)(kRowLds<NS> * kRows));
    if constexpr (sizeof(T) == 2 || NS == 1) {
        if (e == hipSuccess)
            e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_attn_tile<T, NS, kTileWaves<NS>>),
                                    hipFuncAttributeMaxDynamicSharedMemorySize, kTileLds<NS>);
    }
    return e;
}
template <typename T>
hipError_t prepare_all() {
    for (hipError_t e : {prepare<T, 1>(), prepare<T, 2>(), prepare<T, 3>(), prepare<T, 4>()})
        if (e != hipSuccess) return e;
    return hipSuccess;
}

}  // namespace

int attn_tile_rows(int dtype, int slabs) {
    if (dtype == kF32) return slabs == 1 ? 32 * kTileWaves<1> : 0;
    return 32 * (slabs == 1 ? kTileWaves<1> : slabs == 2 ? kTileWaves<2> : slabs == 3 ? kTileWaves<3> : kTileWaves<4>);
}

hipError_t attn_prepare() {
    static std::atomic<uint64_t> done{0};  // a bit per device
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
    for (hipError_t x : {prepare_all<float>(), prepare_all<__bf16>(), prepare_all<_Float16>(), prefix_prepare()})
        if (x != hipSuccess) e = x;
    if (e == hipSuccess && dev < 64) done.fetch_or(1ull << dev);
    return e;
}

hipError_t launch_attn(const AttnArgs& a, int dtype, hipStream_t s) {
    if (dtype == kF32) return attn_as<float>(a, s);
    if (dtype == kBF16) return attn_as<__bf16>(a, s);
    return attn_as<_Float16>(a, s);
}

}  // namespace np
