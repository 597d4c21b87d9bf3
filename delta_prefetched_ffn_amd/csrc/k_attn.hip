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
#include "kv_device.hpp"

namespace np {
namespace {

// What differs by the type of q and out. K codes become Op values (exact), q is held as kTerms
// summands of that type: bf16 and fp16 as they are, fp32 as three bf16 summands (8 + 8 + 8 bits:
// exact). P is rounded to fp16 for 16-bit outputs (2^-11 of the value, below the output's own
// rounding for bf16 and equal to it for fp16) and to three bf16 summands (2^-24) for fp32.
template <typename T>
struct Kind;
template <>
struct Kind<__bf16> {
    typedef __bf16 Q;
    typedef _Float16 P;
    static constexpr int kQ = 1, kP = 1;
};
template <>
struct Kind<_Float16> {
    typedef _Float16 Q;
    typedef _Float16 P;
    static constexpr int kQ = 1, kP = 1;
};
template <>
struct Kind<float> {
    typedef __bf16 Q;
    typedef __bf16 P;
    static constexpr int kQ = 3, kP = 3;
};

template <typename E>
struct Vec8;
template <>
struct Vec8<__bf16> {
    typedef bf16x8 t;
};
template <>
struct Vec8<_Float16> {
    typedef f16x8 t;
};

__device__ inline f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ inline f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// Eight e4m3 codes (two dwords) times 2^k (s = 2^k as a float) to eight 16-bit floats: exact in
// bf16, exact in fp16 while the product stays within its normal range.
template <typename E>
__device__ inline typename Vec8<E>::t widen(uint32_t a, uint32_t b, float s);
template <>
__device__ inline bf16x8 widen<__bf16>(uint32_t a, uint32_t b, float s) {
    const bf16x2 x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, false), y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, true);
    const bf16x2 z = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, false), w = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, true);
    return bf16x8{x[0], x[1], y[0], y[1], z[0], z[1], w[0], w[1]};
}
template <>
__device__ inline f16x8 widen<_Float16>(uint32_t a, uint32_t b, float s) {
    const f16x2 x = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, s, false), y = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, s, true);
    const f16x2 z = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, s, false), w = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, s, true);
    return f16x8{x[0], x[1], y[0], y[1], z[0], z[1], w[0], w[1]};
}

// x[8] as `N` summands of type E, each the rounding of what the ones before left.
template <typename E, int N>
__device__ inline void split(typename Vec8<E>::t* o, const float* x) {
    float r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = x[k];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const E e = (E)r[k];
            o[n][k] = e;
            if (n + 1 < N) r[k] = r[k] - (float)e;
        }
}

constexpr int kRows = 16;    // query rows of a tile
constexpr int kPiece = 32;   // tokens of one step
// P's values reach 2^kLazy before the running maximum is raised, so most steps rescale nothing.
constexpr float kLazy = 8.0f;
// O is kept in units of 2^unit; a block's V codes are widened times 2^(ev - unit). Within
// [-kFar, kNear] of the unit every code is a normal fp16 number (2^-9 * 2^-5 = 2^-14 and
// 448 * 2^7 < 65504), so widening is exact; a block further off moves the unit. It moves down by at
// most kDrop from the largest exponent met (O would overflow fp32): blocks below that vanish.
constexpr int kFar = 5, kNear = 7, kDrop = 40;

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

constexpr int kWaves = 4;

// Few rows: one workgroup per (row tile, split of the key axis, kv head). Its four waves take every
// fourth piece of the split and are joined through LDS at the end; splits are joined by k_attn_join.
template <typename T, int NS>
__global__ __launch_bounds__(64 * kWaves) void k_attn_rows(AttnArgs a) {
    typedef Kind<T> Kd;
    typedef typename Kd::Q Q;
    typedef typename Kd::P P;
    typedef typename Vec8<Q>::t Q8;
    typedef typename Vec8<P>::t P8;
    const KvView& kv = a.kv;
    const int b = find_item(a.b, blockIdx.x), h = blockIdx.y;
    const int item = (int)blockIdx.x - a.b.item0[b], rt = item / a.splits, sp = item - rt * a.splits;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int group = kv.n_heads / kv.n_kv, rows = a.b.fresh[b] * group, r0 = rt * kRows;
    const int row = r0 + col;  // (query token, head of the group)
    const bool real = row < rows;
    const int tq = row / group, head = h * group + row - tq * group;
    const int before = a.b.before[b], pos = before + tq;
    const int pos_lo = before + r0 / group, pos_hi = before + min(r0 + kRows - 1, rows - 1) / group;
    const Pieces pc = pieces_of(pos_lo, pos_hi, a.window, a.sinks);
    const int u0 = (int)((int64_t)pc.total * sp / a.splits), u1 = (int)((int64_t)pc.total * (sp + 1) / a.splits);

    Q8 q[NS][2][Kd::kQ];
#pragma unroll
    for (int c = 0; c < NS; ++c)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const int d = c * 64 + quad * 16 + f * 8;
            float x[8] = {};
            if (real && d < kv.hd)
                load_row<8>(x, static_cast<const T*>(a.q) + (int64_t)(a.b.row0[b] + tq) * a.q_row + (int64_t)head * a.q_head + d);
            split<Q, Kd::kQ>(q[c][f], x);
        }

    const uint8_t* const codes = kv.codes + a.layer * kv.layer_bytes;
    const int8_t* const exps = kv.exps + (int64_t)a.layer * kv.n_pages * kv.n_kv * 2;
    const int side_bytes = (1 << kv.page_shift) * kv.slabs * kTileDims;
    const int seq = a.b.seq[b];

    f32x4 o[NS][4];
#pragma unroll
    for (int c = 0; c < NS; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[c][i] = f32x4{0, 0, 0, 0};
    float m = -__builtin_inff(), l = 0.0f;  // l: this lane's tokens only, joined at the end
    bool seen = false;
    int unit = 0, top = 0;  // o is in units of 2^unit
    bool begun = false;

    for (int u = u0 + wave; u < u1; u += kWaves) {
        const int tok = pc[u] * kPiece;
        u32x4 k[2][NS], v[2][NS];
        float kf[2];
        int ev[2];
        bool held[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int t = tok + 16 * g;
            const int page = t <= pos_hi ? __builtin_amdgcn_readfirstlane(page_of(kv, seq, t >> kv.page_shift)) : -1;
            held[g] = page >= 0;
            kf[g] = 0.0f;
            ev[g] = unit;
            if (held[g]) {
                const int8_t* const e = exps + ((int64_t)page * kv.n_kv + h) * 2;
                kf[g] = a.scale2 * pow2i(max(-126, (int)e[0]));
                ev[g] = max(-126, (int)e[1]);
                const uint8_t* const p = codes + page * kv.page_bytes + (int64_t)h * 2 * side_bytes +
                                         (int64_t)((t & ((1 << kv.page_shift) - 1)) >> 4) * (kv.slabs * kTileBytes) + lane * 16;
#pragma unroll
                for (int c = 0; c < NS; ++c) {
                    k[g][c] = *reinterpret_cast<const u32x4*>(p + c * kTileBytes);
                    v[g][c] = *reinterpret_cast<const u32x4*>(p + side_bytes + c * kTileBytes);
                }
            } else {
#pragma unroll
                for (int c = 0; c < NS; ++c) k[g][c] = v[g][c] = u32x4{0, 0, 0, 0};
            }
        }
        if (!held[0] && !held[1]) continue;

        float s[8];  // tokens tok + 16 (k / 4) + 4 quad + k % 4
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            f32x4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < NS; ++c)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const Q8 kk = widen<Q>(k[g][c][2 * f], k[g][c][2 * f + 1], 1.0f);
#pragma unroll
                    for (int n = 0; n < Kd::kQ; ++n) acc = mfma(kk, q[c][f][n], acc);
                }
#pragma unroll
            for (int j = 0; j < 4; ++j) s[4 * g + j] = acc[j] * kf[g];
        }

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
        const float m0 = m == -__builtin_inff() ? 0.0f : m;  // a row that has seen nothing finite
        float p[8];
#pragma unroll
        for (int k8 = 0; k8 < 8; ++k8) {
            p[k8] = __builtin_amdgcn_exp2f(s[k8] - m0);
            if (!(vis >> k8 & 1)) p[k8] = 0.0f;
            l += p[k8];
        }

        // Normally one pass; two where the groups' V scales lie too far apart for one unit.
        const bool near = !held[0] || !held[1] || (ev[0] - ev[1] <= kNear + kFar && ev[1] - ev[0] <= kNear + kFar);
        for (int pass = 0; pass < (near ? 1 : 2); ++pass) {
            const int e0 = near ? held[0] ? ev[0] : ev[1] : ev[pass], e1 = near ? held[1] ? ev[1] : ev[0] : ev[pass];
            const int lo_e = min(e0, e1), hi_e = max(e0, e1);
            if (!begun) {
                unit = top = min(hi_e, lo_e + kFar);
                begun = true;
            }
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
            float pp[8];
#pragma unroll
            for (int k8 = 0; k8 < 8; ++k8) pp[k8] = near || (k8 >> 2) == pass ? p[k8] : 0.0f;
            P8 pv[Kd::kP];
            split<P, Kd::kP>(pv, pp);
            // Of two passes each takes one group: the other's codes are out (they would overflow at this unit).
            const float f0 = pow2i(max(-126, e0 - unit)), f1 = pow2i(max(-126, e1 - unit));
            const uint32_t in0 = near || pass == 0 ? ~0u : 0u, in1 = near || pass == 1 ? ~0u : 0u;
#pragma unroll
            for (int c = 0; c < NS; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w0 = v[0][c][i] & in0, w1 = v[1][c][i] & in1;
                    uint32_t bad = 0;
                    if (!whole) {
                        // NaN codes of tokens that a row does not see (values that were NaN, or bytes never
                        // written) must not reach it: 0 * NaN is NaN. They are taken out of the product and
                        // given back below to the rows that do see them.
                        const uint32_t n0 = nan_bytes(w0) >> 7, n1 = nan_bytes(w1) >> 7;
                        bad = n0 | n1;
                        w0 &= ~(n0 * 255u);
                        w1 &= ~(n1 * 255u);
                        if (__any(bad)) {
                            const P8 ones = widen<P>(n0 * 0x38u, n1 * 0x38u, 1.0f);  // 0x38 is 1.0
                            float see[8];
#pragma unroll
                            for (int k8 = 0; k8 < 8; ++k8) see[k8] = vis >> k8 & 1 ? 1.0f : 0.0f;
                            P8 sv[1];
                            split<P, 1>(sv, see);
                            const f32x4 hit = mfma(ones, sv[0], f32x4{0, 0, 0, 0});
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (hit[j] > 0.0f) o[c][i][j] = __builtin_nanf("");
                        }
                    }
                    // widen's dwords: four tokens of group 0, four of group 1
                    P8 vv;
                    if (f0 == f1) {
                        vv = widen<P>(w0, w1, f0);
                    } else {
                        const P8 x0 = widen<P>(w0, w0, f0), x1 = widen<P>(w1, w1, f1);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            vv[j] = x0[j];
                            vv[4 + j] = x1[j];
                        }
                    }
#pragma unroll
                    for (int n = 0; n < Kd::kP; ++n) o[c][i] = mfma(vv, pv[n], o[c][i]);
                }
        }
    }

    // Join the waves: rows' maximum, sum and O in true units.
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    seen = (__ballot(seen) >> col & 0x0001000100010001ull) != 0;
    if (seen && m == -__builtin_inff()) l = __builtin_nanf("");  // every visible score is -inf: 0 / 0
    constexpr int D = NS * 64;
    __shared__ float s_o[kWaves][kRows][D + 4], s_m[kWaves][kRows], s_l[kWaves][kRows];
    const float back = pow2i(max(-126, min(127, unit)));
#pragma unroll
    for (int c = 0; c < NS; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s_o[wave][col][c * 64 + quad * 16 + 4 * j + i] = o[c][i][j] * back;
    if (quad == 0) {
        s_m[wave][col] = m;
        s_l[wave][col] = l;
    }
    __syncthreads();
    const int D4 = kv.hd / 4;
    for (int k = threadIdx.x; k < kRows * D4; k += 64 * kWaves) {
        const int r = k / D4, d = (k - r * D4) * 4;
        if (r0 + r >= rows) break;
        float mm = s_m[0][r], ll = 0.0f;
#pragma unroll
        for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, s_m[w][r]);
        f32x4 x = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = s_m[w][r] == mm ? 1.0f : __builtin_amdgcn_exp2f(s_m[w][r] - mm);
            if (s_l[w][r] == 0.0f && f == 1.0f && s_m[w][r] == -__builtin_inff()) continue;  // saw nothing
            ll += f * s_l[w][r];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] += f * s_o[w][r][d + j];
        }
        const bool none = mm == -__builtin_inff() && ll == 0.0f;  // no visible token: 0
        const int t = (r0 + r) / group, hd = h * group + (r0 + r) - t * group;
        if (a.splits == 1) {
            T* const out = static_cast<T*>(a.out) + (int64_t)(a.b.row0[b] + t) * a.o_row + (int64_t)hd * a.o_head + d;
#pragma unroll
            for (int j = 0; j < 4; ++j) out[j] = (T)(none ? 0.0f : x[j] / ll);
            if (a.lse && d == 0)
                a.lse[(int64_t)(a.b.row0[b] + t) * kv.n_heads + hd] = none ? -__builtin_inff() : (mm + log2f(ll)) * 0.69314718055994531f;
        } else {
            float* const part = a.part + (((int64_t)blockIdx.x * kv.n_kv + h) * kRows + r) * (D + 2);
#pragma unroll
            for (int j = 0; j < 4; ++j) part[2 + d + j] = x[j];
            if (d == 0) {
                part[0] = mm;
                part[1] = ll;
            }
        }
    }
}

// Joins the splits of a row tile, in order: one workgroup per (row tile, kv head).
template <typename T>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
    const KvView& kv = a.kv;
    const int first = (int)blockIdx.x * a.splits;
    const int b = find_item(a.b, first), h = blockIdx.y;
    const int rt = (first - a.b.item0[b]) / a.splits;
    const int group = kv.n_heads / kv.n_kv, rows = a.b.fresh[b] * group, r0 = rt * kRows, D = kv.slabs * 64, D4 = kv.hd / 4;
    for (int k = threadIdx.x; k < kRows * D4; k += 256) {
        const int r = k / D4, d = (k - r * D4) * 4;
        if (r0 + r >= rows) break;
        const int64_t stride = (int64_t)kv.n_kv * kRows * (D + 2);
        const float* const p = a.part + (((int64_t)first * kv.n_kv + h) * kRows + r) * (D + 2);
        float mm = -__builtin_inff(), ll = 0.0f;
        for (int s = 0; s < a.splits; ++s) mm = fmaxf(mm, p[s * stride]);
        f32x4 x = {0, 0, 0, 0};
        for (int s = 0; s < a.splits; ++s) {
            const float ms = p[s * stride], ls = p[s * stride + 1];
            if (ms == -__builtin_inff() && ls == 0.0f) continue;  // saw nothing
            const float f = ms == mm ? 1.0f : __builtin_amdgcn_exp2f(ms - mm);
            ll += f * ls;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] += f * p[s * stride + 2 + d + j];
        }
        const bool none = mm == -__builtin_inff() && ll == 0.0f;
        const int t = (r0 + r) / group, hd = h * group + (r0 + r) - t * group;
        T* const out = static_cast<T*>(a.out) + (int64_t)(a.b.row0[b] + t) * a.o_row + (int64_t)hd * a.o_head + d;
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = (T)(none ? 0.0f : x[j] / ll);
        if (a.lse && d == 0)
            a.lse[(int64_t)(a.b.row0[b] + t) * kv.n_heads + hd] = none ? -__builtin_inff() : (mm + log2f(ll)) * 0.69314718055994531f;
    }
}

template <typename T>
hipError_t rows_as(const AttnArgs& a, hipStream_t s) {
    const dim3 grid(a.b.item0[a.b.n], a.kv.n_kv);
    switch (a.kv.slabs) {
        case 1: k_attn_rows<T, 1><<<grid, 64 * kWaves, 0, s>>>(a); break;
        case 2: k_attn_rows<T, 2><<<grid, 64 * kWaves, 0, s>>>(a); break;
        case 3: k_attn_rows<T, 3><<<grid, 64 * kWaves, 0, s>>>(a); break;
        default: k_attn_rows<T, 4><<<grid, 64 * kWaves, 0, s>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, int dtype, hipStream_t s) {
    if (dtype == kF32) return rows_as<float>(a, s);
    if (dtype == kBF16) return rows_as<__bf16>(a, s);
    return rows_as<_Float16>(a, s);
}

hipError_t launch_attn_join(const AttnArgs& a, int dtype, hipStream_t s) {
    const dim3 grid(a.b.item0[a.b.n] / a.splits, a.kv.n_kv);
    if (dtype == kF32) k_attn_join<float><<<grid, 256, 0, s>>>(a);
    else if (dtype == kBF16) k_attn_join<__bf16><<<grid, 256, 0, s>>>(a);
    else k_attn_join<_Float16><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace np
