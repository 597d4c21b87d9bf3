// Products with 4-bit weights for gfx950 (semantics: include/np.h):
//     y[r][o] = sum_i s[o][g(i)] * (c[o][i] - z[o][g(i)]) * x[r][i].
//
// A code c in 0 .. 15, as a byte, is the e4m3 number c * 2^-9 (its lowest numbers are equidistant), so the conversion
// instruction that the attention uses makes two 16-bit operands of two codes, exactly, with nothing to subtract. The zero
// point leaves the product: per group, sum (c - z) x = sum c x - z sum x, whose second sum comes from a product with ones;
// both are fp32 sums of at most `group` terms. The scales multiply these sums in fp32, so no weight is rounded.
//
// Rows of x that hold infinities, or sums that overflow, would give inf - inf there: lanes that end with a sum that is not
// finite work it out again with operands c - z (exact, and slower).
#include <algorithm>
#include <atomic>

#include "mfma_device.hpp"
#include "w4_internal.hpp"

namespace np {
namespace {

// What differs by the type of x: the operands, and how many of them sum up to one value (fp32: three of 8 bits, exact).
template <typename T>
struct Kind;
template <>
struct Kind<__bf16> {
    typedef __bf16 E;
    static constexpr int kTerms = 1;
};
template <>
struct Kind<_Float16> {
    typedef _Float16 E;
    static constexpr int kTerms = 1;
};
template <>
struct Kind<float> {
    typedef __bf16 E;
    static constexpr int kTerms = 3;
};

// Eight codes (one dword of a tile) as operands.
template <typename E>
__device__ inline typename Vec8<E>::t codes_of(uint32_t w) {
    return widen<E>(w & 0x0f0f0f0fu, w >> 4 & 0x0f0f0f0fu, 512.0f, 512.0f);
}
// The same less z.
template <typename E>
__device__ inline typename Vec8<E>::t weights_of(uint32_t w, int z) {
    typename Vec8<E>::t o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = (E)(float)((int)(w >> ((j & 3) * 8 + (j >> 2) * 4) & 15) - z);
    return o;
}
template <typename E>
__device__ inline typename Vec8<E>::t ones() {
    typename Vec8<E>::t o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = (E)1.0f;
    return o;
}

// A group's scale and zero point, as they are loaded, and their values.
struct __attribute__((packed, aligned(4))) ScaleWords {
    uint32_t w[2];
};
__device__ inline u32x2 load_scale(const W4View& w, int64_t at) {
    const ScaleWords s = *reinterpret_cast<const ScaleWords*>(w.scales + at * w.scale_words);
    return u32x2{s.w[0], s.w[1]};
}
__device__ inline float scale_value(u32x2 s, int words) { return __uint_as_float(s[0] & (words == 1 ? ~15u : ~0u)); }
__device__ inline int zero_value(u32x2 s, int words) { return (int)((words == 1 ? s[0] : s[1]) & 15); }

// y = v, or y + v, rounded once.
__device__ inline void put(const W4Args& a, int64_t row, int out, float v) {
    const int64_t at = row * a.y_row + out;
    if (a.y_dtype == 0) {
        float* const y = static_cast<float*>(a.y) + at;
        *y = a.accumulate ? *y + v : v;
    } else if (a.y_dtype == 1) {
        __bf16* const y = static_cast<__bf16*>(a.y) + at;
        *y = (__bf16)(a.accumulate ? (float)*y + v : v);
    } else {
        _Float16* const y = static_cast<_Float16*>(a.y) + at;
        *y = (_Float16)(a.accumulate ? (float)*y + v : v);
    }
}

__device__ inline bool not_finite(float x) { return !(fabsf(x) <= __FLT_MAX__); }

// Eight values of x as operands: 16 bits a value as they are, fp32 split.
template <typename T>
struct XRaw {
    u32x4 v[sizeof(T) / 2];
};
template <typename T>
__device__ inline XRaw<T> load_x(const T* p, bool in) {
    XRaw<T> r;
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) r.v[k] = in ? reinterpret_cast<const u32x4*>(p)[k] : u32x4{0, 0, 0, 0};
    return r;
}
template <typename T>
__device__ inline void operands(typename Vec8<typename Kind<T>::E>::t* o, const XRaw<T>& r) {
    typedef typename Kind<T>::E E;
    if constexpr (sizeof(T) == 2) {
        o[0] = __builtin_bit_cast(typename Vec8<E>::t, r.v[0]);
    } else {
        // Leading bits first: what a term leaves is exact. (An infinity leaves NaN, which ends in a sum that is not finite.)
        float x[8];
        __builtin_memcpy(x, r.v, sizeof x);
#pragma unroll
        for (int n = 0; n < Kind<T>::kTerms; ++n)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t u = __float_as_uint(x[k]) & 0xffff0000u;
                o[n][k] = __builtin_bit_cast(__bf16, (uint16_t)(u >> 16));
                x[k] -= __uint_as_float(u);
            }
    }
}
// The same with infinities and NaN as themselves.
template <typename T>
__device__ inline void operands_of_any(typename Vec8<typename Kind<T>::E>::t* o, const XRaw<T>& r) {
    operands<T>(o, r);
    if constexpr (sizeof(T) == 4) {
        float x[8];
        __builtin_memcpy(x, r.v, sizeof x);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (!not_finite(x[k])) continue;
            o[0][k] = (__bf16)x[k];
            o[1][k] = o[2][k] = (__bf16)0.0f;
        }
    }
}

constexpr int kWaves = 8;

// Few rows: one workgroup per 16 O outputs and 16 R rows; its waves take every kWaves-th chunk of 128 inputs and are joined
// in LDS, in their order. A lane's 16 bytes of a tile are its operands of four products, x the other one: D row = row of x,
// D column = output. x comes from the caches, once for O tiles (kStaged: fp32, split once per workgroup into LDS). U chunks are on
// their way at a time.
//
// Bound by the weights' way from memory at first: one row of 4096 x 11008 takes 7.6 us (3.1 TB/s), of 32,000 x 4096 13.3 us (5.1 TB/s;
// 25 us before O went up to 4, since every workgroup reads all of x), with the empty launch's 3.5. With more rows x itself comes first:
// every workgroup reads all its rows of it from the caches, 64 rows of 4096 x 4096 134 MB in 18 us, 128 rows of 4096 x 11008 0.72 GB
// in 82 us (8.8 TB/s).
template <typename T, int R, int O, int U, bool kStaged, int G>
__global__ __launch_bounds__(64 * kWaves, R == 1 ? 4 : 2) void k_w4_rows(W4Args a) {
    typedef Kind<T> Kd;
    typedef typename Kd::E E;
    typedef typename Vec8<E>::t E8;
    constexpr int N = Kd::kTerms, kStride = kW4Outs * O + 1;
    const W4View& w = a.w;
    const int tile0 = blockIdx.x * O, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int64_t r0 = (int64_t)blockIdx.y * 16 * R;
    const int rows = (int)min((int64_t)16 * R, a.rows - r0);
    extern __shared__ __attribute__((aligned(128))) uint8_t s_dyn[];
    E* const s_x = reinterpret_cast<E*>(s_dyn);              // [N][rows][x_len]
    float* const s_part = reinterpret_cast<float*>(s_dyn);   // [waves][16 R][kStride], behind the products
    const int x_len = w.chunks * kW4Ins + 8;

    // Rows past the last read the last one, tiles past the last the last one: what they give is not stored.
    const T* xr[R];
#pragma unroll
    for (int r = 0; r < R; ++r) xr[r] = static_cast<const T*>(a.x) + (r0 + min(16 * r + col, rows - 1)) * a.x_row + quad * 8;
    int tile[O];
#pragma unroll
    for (int o = 0; o < O; ++o) tile[o] = min(tile0 + o, w.out_tiles - 1);

    struct Part {
        u32x4 code[O];
        XRaw<T> x[kStaged ? 1 : R][4];
        u32x2 scale[O][G];
    };
    const auto ask = [&](Part& p, int c) __attribute__((always_inline)) {
#pragma unroll
        for (int o = 0; o < O; ++o) p.code[o] = *reinterpret_cast<const u32x4*>(w.tiles + ((int64_t)tile[o] * w.chunks + c) * kW4TileBytes + lane * 16);
        if constexpr (!kStaged) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int s = 0; s < 4; ++s) p.x[r][s] = load_x<T>(xr[r] + c * kW4Ins + s * 32, c * kW4Ins + s * 32 + quad * 8 < w.n_in);
        }
#pragma unroll
        for (int o = 0; o < O; ++o)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int64_t at = (((int64_t)tile[o] * w.chunks + c) * G + g) * kW4Outs + col;
                p.scale[o][g] = load_scale(w, at);
            }
    };
    const auto x_of = [&](E8* o, const Part& p, int c, int r, int s) __attribute__((always_inline)) {
        if constexpr (kStaged) {
#pragma unroll
            for (int n = 0; n < N; ++n)
                o[n] = *reinterpret_cast<const E8*>(s_x + (int64_t)(n * rows + min(col, rows - 1)) * x_len + c * kW4Ins + s * 32 + quad * 8);
        } else {
            operands<T>(o, p.x[r][s]);
        }
    };
    f32x4 tot[R][O];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int o = 0; o < O; ++o) tot[r][o] = f32x4{0, 0, 0, 0};
    const auto products = [&](const Part& p, int c) __attribute__((always_inline)) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            f32x4 part[R][O], sum[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                sum[r] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int o = 0; o < O; ++o) part[r][o] = f32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int s = g * 4 / G; s < (g + 1) * 4 / G; ++s) {
                E8 cw[O];
#pragma unroll
                for (int o = 0; o < O; ++o) cw[o] = codes_of<E>(p.code[o][s]);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    E8 x[N];
                    x_of(x, p, c, r, s);
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        sum[r] = mfma(x[n], ones<E>(), sum[r]);
#pragma unroll
                        for (int o = 0; o < O; ++o) part[r][o] = mfma(x[n], cw[o], part[r][o]);
                    }
                }
            }
#pragma unroll
            for (int o = 0; o < O; ++o) {
                const float sc = scale_value(p.scale[o][g], w.scale_words), z = (float)zero_value(p.scale[o][g], w.scale_words);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int j = 0; j < 4; ++j) tot[r][o][j] = __builtin_fmaf(sc, __builtin_fmaf(-z, sum[r][j], part[r][o][j]), tot[r][o][j]);
#pragma unroll
                for (int r = 0; r < R; ++r) asm volatile("" : "+v"(tot[r][o]));  // here, not behind the loads to come
            }
        }
    };

    Part ring[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (wave + u * kWaves < w.chunks) ask(ring[u], wave + u * kWaves);
    if constexpr (kStaged) {
        const int units = w.chunks * (kW4Ins / 8);  // eight values each
        for (int i = threadIdx.x; i < rows * units; i += 64 * kWaves) {
            const int r = i / units, k = (i - r * units) * 8;
            const XRaw<T> raw = load_x<T>(static_cast<const T*>(a.x) + (r0 + r) * a.x_row + k, k < w.n_in);
            E8 o[N];
            operands<T>(o, raw);
#pragma unroll
            for (int n = 0; n < N; ++n) *reinterpret_cast<E8*>(s_x + (int64_t)(n * rows + r) * x_len + k) = o[n];
        }
        __syncthreads();
    }
    for (int c = wave; c < w.chunks; c += kWaves * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = c + u * kWaves;
            if (at >= w.chunks) break;
            products(ring[u], at);
            if (at + U * kWaves < w.chunks) ask(ring[u], at + U * kWaves);
        }
    }
    bool odd = false;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int o = 0; o < O; ++o)
#pragma unroll
            for (int j = 0; j < 4; ++j) odd |= not_finite(tot[r][o][j]);
    if (__any(odd)) {
        // The wave's products again, one at a time.
#pragma unroll 1
        for (int ro = 0; ro < R * O; ++ro) {
            const int r = ro / O, t = min(tile0 + ro - r * O, w.out_tiles - 1);
            const T* const x0 = static_cast<const T*>(a.x) + (r0 + min(16 * r + col, rows - 1)) * a.x_row;
            f32x4 again = {0, 0, 0, 0};
#pragma unroll 1
            for (int c = wave; c < w.chunks; c += kWaves) {
                const u32x4 code = *reinterpret_cast<const u32x4*>(w.tiles + ((int64_t)t * w.chunks + c) * kW4TileBytes + lane * 16);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int64_t at = (((int64_t)t * w.chunks + c) * G + s * G / 4) * kW4Outs + col;
                    const u32x2 words = load_scale(w, at);
                    const float sc = scale_value(words, w.scale_words);
                    const E8 cw = weights_of<E>(code[s], zero_value(words, w.scale_words));
                    const int k = c * kW4Ins + s * 32 + quad * 8;
                    E8 x[N];
                    operands_of_any<T>(x, load_x<T>(x0 + k, k < w.n_in));
                    f32x4 part = {0, 0, 0, 0};
#pragma unroll
                    for (int n = 0; n < N; ++n) part = mfma(x[n], cw, part);
#pragma unroll
                    for (int j = 0; j < 4; ++j) again[j] = __builtin_fmaf(sc, part[j], again[j]);
                }
            }
#pragma unroll
            for (int i = 0; i < R * O; ++i)
                if (i == ro)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (not_finite(tot[i / O][i % O][j])) tot[i / O][i % O][j] = again[j];
        }
    }
    if (kStaged) __syncthreads();  // x is done with
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int o = 0; o < O; ++o)
#pragma unroll
            for (int j = 0; j < 4; ++j) s_part[(wave * 16 * R + 16 * r + 4 * quad + j) * kStride + kW4Outs * o + col] = tot[r][o][j];
    __syncthreads();
    for (int i = threadIdx.x; i < rows * kW4Outs * O; i += 64 * kWaves) {
        const int r = i / (kW4Outs * O), out = i % (kW4Outs * O);
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) v += s_part[(k * 16 * R + r) * kStride + out];
        if (tile0 * kW4Outs + out < w.n_out) put(a, r0 + r, tile0 * kW4Outs + out, v);
    }
}

// Many rows: one workgroup of 4 S waves per (64 H rows, 128 outputs); a wave has all the rows x 32 outputs, in products of
// 32x32x16, S = 2 of them half of each chunk's inputs each, joined in LDS behind the last one. The workgroup's x of a chunk of 128 inputs
// is in LDS as operands (two chunks: one is read while the next one's loads are on their way), with the sums of each row and group (or half
// of one), three bf16 terms of them, that take the zero points out: one more product per group, with -z as the other operand. Each wave
// widens the codes of its outputs itself, no two the same ones.
//
// Bound by waiting, at two waves a SIMD: a wave waits for data and barriers for 0.43 of its time and for its turn to issue for 0.21; the
// matrix units are busy for 0.36 of theirs, other vector instructions (302 a wave and chunk beside 36 products) take 0.38. 1,500 rows x 5120 x
// 15,360 (H = 2, S = 1): 325 us in bf16 (726 TFLOP/s), with groups of 32 429 us; with waves of half the rows x 64 outputs, which widen all
// codes twice, 345 and 481 us. fp32 (H = 1, S = 2; three products for each) 1,058 us.
//
// Operand slots: step (s, e) of a chunk, lane half h: inputs 32 s + 8 (h + 2 e) + j, so that a lane's 16 bytes of quad h + 2 e of a
// tile are its operands of four steps.
constexpr int kTileOuts = 128;

template <typename T>
__device__ inline float sum8(const XRaw<T>& r) {
    float v = 0.0f;
    if constexpr (sizeof(T) == 4) {
        float x[8];
        __builtin_memcpy(x, r.v, sizeof x);
        v = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t u = r.v[0][k];  // a bit cast of the vector's element itself would take the first one
            if constexpr (__is_same(T, __bf16)) v = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, u), bf16x2{(__bf16)1.0f, (__bf16)1.0f}, v, false);
            else v = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, u), f16x2{(_Float16)1.0f, (_Float16)1.0f}, v, false);
        }
    }
    return v;
}
// x summed over the lanes of its four neighbours.
__device__ inline float quad_sum(float x) {
    x += __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0xb1, 0xf, 0xf, true));  // 1 0 3 2
    x += __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0x4e, 0xf, 0xf, true));  // 2 3 0 1
    return x;
}

template <typename T, int H, int S, int G>
__global__ __launch_bounds__(256 * S, S == 1 ? 2 : sizeof(T) == 2 && G < 4 ? 4 : 2) void k_w4_tile(W4Args a, int row_blocks, int out_blocks) {
    typedef Kind<T> Kd;
    typedef typename Kd::E E;
    typedef typename Vec8<E>::t E8;
    constexpr int N = Kd::kTerms, kRows = 64 * H, RT = 2 * H, TT = 1, SG = G < S ? S : G;
    static_assert(H * S <= 2, "a wave stages whole rows or half chunks of them");
    const W4View& w = a.w;
    // Workgroups go to the 8 dies in turn: a die takes its own outputs, with all rows one after the other.
    const int die = blockIdx.x & 7, nth = blockIdx.x >> 3;
    const int ob = die + 8 * (nth / row_blocks), rb = nth % row_blocks;
    if (ob >= out_blocks) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int64_t r0 = (int64_t)rb * kRows;
    const int rows = (int)min((int64_t)kRows, a.rows - r0);
    const int part_of = wave >> 2, tile0 = ob * 8 + (wave & 3) * 2;
    extern __shared__ __attribute__((aligned(128))) uint8_t s_dyn[];
    E8* const s_x = reinterpret_cast<E8*>(s_dyn);  // [2][2 H row tiles][8 steps][N][2 halves][32 rows, changed places]
    constexpr int kBuf = 2 * H * 8 * N * 64;
    bf16x8* const s_sum = reinterpret_cast<bf16x8*>(s_dyn + 2 * kBuf * 16);  // [2][SG][rows]

    // Staging: a wave brings 16 H rows in units of 16 rows x 32 inputs: lane 4 r + q has quad q of row r. Places in LDS: row r of (step,
    // half) at r ^ 4 q, so that a unit's 64 stores meet no bank twice.
    constexpr int kSteps = 4 / S;  // of 32 inputs, that a wave brings
    XRaw<T> stage[H][kSteps];
    const int sr = lane >> 2, sq = lane & 3;
    const T* xs[H];
#pragma unroll
    for (int u = 0; u < H; ++u) xs[u] = static_cast<const T*>(a.x) + (r0 + min((wave & 3) * 16 * H + u * 16 + sr, rows - 1)) * a.x_row + part_of * kSteps * 32 + sq * 8;
    const auto ask_x = [&](int c) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < H; ++u)
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                stage[u][s] = load_x<T>(xs[u] + c * kW4Ins + s * 32, c * kW4Ins + (part_of * kSteps + s) * 32 + sq * 8 < w.n_in);
    };
    const auto put_x = [&](int c) __attribute__((always_inline)) {
        E8* const to = s_x + (c & 1) * kBuf;
        bf16x8* const sums = s_sum + (c & 1) * SG * kRows;
#pragma unroll
        for (int u = 0; u < H; ++u) {
            const int row = (wave & 3) * 16 * H + u * 16 + sr;
            float part[kSteps];
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                E8 o[N];
                operands<T>(o, stage[u][s]);
#pragma unroll
                for (int n = 0; n < N; ++n)
                    to[((((row >> 5) * 8 + 2 * (part_of * kSteps + s) + (sq >> 1)) * N + n) * 2 + (sq & 1)) * 32 + ((row & 31) ^ (4 * sq))] = o[n];
                part[s] = quad_sum(sum8<T>(stage[u][s]));
            }
            // Lane q writes the sum of the wave's group q.
            constexpr int kSums = SG / S;
            float v = part[0];
            if constexpr (kSums == 4) v = sq == 0 ? part[0] : sq == 1 ? part[1] : sq == 2 ? part[2] : part[3];
            else if constexpr (kSums == kSteps) v = sq ? part[1] : part[0];
            else if constexpr (kSums == 2) v = sq ? part[2] + part[3] : part[0] + part[1];
            else if constexpr (kSteps == 2) v = part[0] + part[1];
            else v = (part[0] + part[1]) + (part[2] + part[3]);
            u32x4 t = {0, 0, 0, 0};
            const uint32_t t0 = __float_as_uint(v) & 0xffff0000u;
            v -= __uint_as_float(t0);
            const uint32_t t1 = __float_as_uint(v) & 0xffff0000u;
            v -= __uint_as_float(t1);
            t[0] = t0 >> 16 | t1;
            t[1] = __float_as_uint(v) >> 16;
            if (sq < kSums) sums[(part_of * kSums + sq) * kRows + row] = __builtin_bit_cast(bf16x8, t);
        }
    };
    // Codes of outputs 32 t + col: quads h and h + 2 of the tile.
    const uint8_t* tiles[TT];
    int64_t groups[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int64_t tile = min(tile0 + 2 * t + (col >> 4), w.out_tiles - 1);  // past the last: not stored
        tiles[t] = w.tiles + tile * w.chunks * kW4TileBytes + (h * 16 + (col & 15)) * 16 + part_of * kSteps * 4;
        groups[t] = tile * w.chunks * G * kW4Outs + (col & 15);
    }
    // Of a chunk's SG parts (groups, or halves of one) a wave takes kParts, and the dwords of its steps.
    constexpr int kParts = SG / S;
    struct Codes {
        alignas(4 * kSteps) uint32_t s[kSteps];
    };
    Codes code[TT][2], next[TT][2];
    u32x2 scale[TT][kParts];
    const auto ask_codes = [&](Codes (&o)[TT][2], int c) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) o[t][e] = *reinterpret_cast<const Codes*>(tiles[t] + (int64_t)c * kW4TileBytes + e * 512);
    };
    const auto ask_scales = [&](int c) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int g = 0; g < kParts; ++g) {
                const int64_t at = groups[t] + (c * G + (part_of * kParts + g) * G / SG) * kW4Outs;
                scale[t][g] = load_scale(w, at);
            }
    };
    float tot[RT][TT][16];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) tot[r][t][j] = 0.0f;

    ask_x(0);
    ask_codes(code, 0);
    put_x(0);
    for (int c = 0; c < w.chunks; ++c) {
        __syncthreads();
        ask_scales(c);  // used behind the first group's products
        if (c + 1 < w.chunks) {
            ask_x(c + 1);
            ask_codes(next, c + 1);
        }
        const E8* const from = s_x + (c & 1) * kBuf + h * 32;
        const bf16x8* const sums = s_sum + (c & 1) * SG * kRows + col;
#pragma unroll
        for (int g = 0; g < kParts; ++g) {
            f32x16 part[RT][TT];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[r][t][j] = 0.0f;
#pragma unroll
            for (int at = 0; at < 8 / SG; ++at) {
                const int own = g * (8 / SG) + at, step = part_of * 2 * kSteps + own, s = own >> 1, e = own & 1;
                E8 cw[TT];
#pragma unroll
                for (int t = 0; t < TT; ++t) cw[t] = codes_of<E>(code[t][e].s[s]);
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const E8 x = from[((r * 8 + step) * N + n) * 64 + (col ^ (4 * (h + 2 * e)))];
#pragma unroll
                        for (int t = 0; t < TT; ++t) part[r][t] = mfma(x, cw[t], part[r][t]);
                    }
            }
            bf16x8 xs8[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) xs8[r] = sums[(part_of * kParts + g) * kRows + 32 * r];
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const float sc = scale_value(scale[t][g], w.scale_words), z = (float)zero_value(scale[t][g], w.scale_words);
                const uint32_t zb = h ? 0u : __float_as_uint(-z);  // whole numbers up to 15: the upper half is bf16
                const bf16x8 minus = __builtin_bit_cast(bf16x8, u32x4{zb >> 16 | zb, zb >> 16, 0, 0});
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    part[r][t] = mfma(xs8[r], minus, part[r][t]);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        tot[r][t][j] = __builtin_fmaf(sc, part[r][t][j], tot[r][t][j]);
                        // Here: the compiler moves these behind the next stores, and all groups' sums wait for them.
                        if constexpr (sizeof(T) == 2) asm volatile("" : "+v"(tot[r][t][j]));
                    }
                }
            }
            if (G > 1) __builtin_amdgcn_sched_barrier(0);
        }
        if (c + 1 < w.chunks) {
            put_x(c + 1);
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) code[t][e] = next[t][e];
        }
    }
    bool odd = false;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) odd |= not_finite(tot[r][t][j]);
    if (__any(odd)) {
        // The wave's products again, one at a time, x from memory.
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const T* const x0 = static_cast<const T*>(a.x) + (r0 + min(32 * r + col, rows - 1)) * a.x_row;
                const int64_t tile = min(tile0 + 2 * t + (col >> 4), w.out_tiles - 1);
                f32x16 again;
#pragma unroll
                for (int j = 0; j < 16; ++j) again[j] = 0.0f;
#pragma unroll 1
                for (int c = 0; c < w.chunks; ++c) {
#pragma unroll 1
                    for (int e = 0; e < 2; ++e) {
                        const int q = h + 2 * e;
                        const uint32_t* const cd = reinterpret_cast<const uint32_t*>(w.tiles + (tile * w.chunks + c) * kW4TileBytes + (q * 16 + (col & 15)) * 16);
#pragma unroll 1
                        for (int s = part_of * kSteps; s < (part_of + 1) * kSteps; ++s) {
                            const int g = s * G / 4, k = c * kW4Ins + s * 32 + q * 8;
                            const int64_t at = ((tile * w.chunks + c) * G + g) * kW4Outs + (col & 15);
                            const u32x2 words = load_scale(w, at);
                            const float sc = scale_value(words, w.scale_words);
                            const E8 cw = weights_of<E>(cd[s], zero_value(words, w.scale_words));
                            E8 x[N];
                            operands_of_any<T>(x, load_x<T>(x0 + k, k < w.n_in));
                            f32x16 part;
#pragma unroll
                            for (int j = 0; j < 16; ++j) part[j] = 0.0f;
#pragma unroll
                            for (int n = 0; n < N; ++n) part = mfma(x[n], cw, part);
#pragma unroll
                            for (int j = 0; j < 16; ++j) again[j] = __builtin_fmaf(sc, part[j], again[j]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (not_finite(tot[r][t][j])) tot[r][t][j] = again[j];
            }
        }
    }
    if constexpr (S > 1) {  // the other half's sums, through LDS
        float* const s_part = reinterpret_cast<float*>(s_dyn);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                float* const at = s_part + ((wave & 3) * RT * 16 + r * 16 + j) * 64 + lane;
                if (part_of) *at = tot[r][0][j];
            }
        __syncthreads();
        if (part_of) return;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < 16; ++j) tot[r][0][j] += s_part[(wave * RT * 16 + r * 16 + j) * 64 + lane];
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int row = 32 * r + 8 * (j >> 2) + 4 * h + (j & 3), tile = tile0 + 2 * t + (col >> 4), out = tile * kW4Outs + (col & 15);
                if (row < rows && out < w.n_out) put(a, r0 + row, out, tot[r][t][j]);
            }
}

// Lays the weights out: a thread per dword of the tiles, and per (group, output).
constexpr int kPackGrid = 1 << 16;
__global__ __launch_bounds__(256) void k_w4_pack(W4PackArgs a) {
    const int64_t tiles = (int64_t)a.out_tiles * a.chunks, step = (int64_t)gridDim.x * 256, first = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t i = first; i < tiles * 256; i += step) {
        const int64_t tile = i >> 8;
        const int lane = (int)(i >> 2) & 63, s = (int)i & 3;
        const int out = (int)(tile / a.chunks) * kW4Outs + (lane & 15), k = (int)(tile % a.chunks) * kW4Ins + s * 32 + (lane >> 4) * 8;
        uint32_t w = 0;
        if (out < a.n_out && k < a.n_in) {
            const uint32_t from = *reinterpret_cast<const uint32_t*>(a.codes + ((int64_t)out * a.n_in + k) / 2);
#pragma unroll
            for (int j = 0; j < 4; ++j) w |= (from >> (4 * j) & 15) << (8 * j) | (from >> (16 + 4 * j) & 15) << (8 * j + 4);
        }
        reinterpret_cast<uint32_t*>(a.tiles)[i] = w;
    }
    for (int64_t i = first; i < tiles * a.per_chunk * kW4Outs; i += step) {
        const int64_t at = i / kW4Outs, all = (int64_t)a.chunks * a.per_chunk;  // at: (tile, chunk, group of the chunk)
        const int out = (int)(at / all) * kW4Outs + (int)(i % kW4Outs), k = (int)(at % all) * (kW4Ins / a.per_chunk);
        const bool in = out < a.n_out && k < a.n_in;
        const int64_t from = (int64_t)out * a.groups + k / a.group;
        const uint32_t z = !in ? 0 : a.zeros ? a.zeros[from] & 15 : 8;
        if (a.scale_dtype == 0) {
            a.scales_out[2 * i] = in ? static_cast<const uint32_t*>(a.scales)[from] : 0;
            a.scales_out[2 * i + 1] = z;
        } else {
            const uint16_t raw = in ? static_cast<const uint16_t*>(a.scales)[from] : 0;
            const uint32_t v = a.scale_dtype == 1 ? (uint32_t)raw << 16 : __float_as_uint((float)__builtin_bit_cast(_Float16, raw));
            a.scales_out[i] = (v & ~15u) | z;
        }
    }
}

// LDS of k_w4_rows: for x, split (fp32), of which it uses at most kStageBytes, then for the waves' results.
constexpr int kStageBytes = 80 * 1024;  // half of a compute unit's
int64_t stage_bytes(const W4Args& a) { return a.rows * (a.w.chunks * kW4Ins + 8) * 3 * 2; }
template <int R, int O>
constexpr int kPartLds = kWaves * 16 * R * (kW4Outs * O + 1) * 4;

// Output tiles of a workgroup, at most, and chunks on their way at a time: what the registers hold of two workgroups a compute
// unit (R = 1) or one.
template <typename T, int R, bool kStaged, int G>
constexpr int kMostO = sizeof(T) == 2 ? (R == 4 || (R == 1 && G > 1) ? 2 : 4) : R == 4 ? 1 : kStaged && G < 4 ? 4 : 2;
template <typename T, int R, int O, bool kStaged, int G>
constexpr int kAhead = sizeof(T) == 4 ? (kStaged && O == 1 ? 2 : 1)
                       : R == 1       ? (O == 4 ? 1 : O == 2 ? (G == 4 ? 1 : 2) : G == 4 ? 2 : 3)
                       : R == 2       ? (O == 4 ? 1 : 2)
                                      : (O == 1 ? 2 : 1);
// As many as leave one workgroup of 64 rows or less for every compute unit.
template <typename T, int R, bool kStaged, int G>
int rows_o(const W4Args& a) {
    return std::min(a.w.out_tiles < 512 ? 1 : a.w.out_tiles < 1024 ? 2 : 4, kMostO<T, R, kStaged, G>);
}
template <typename T, int R, int O, bool kStaged, int G>
constexpr auto* kRowsKernel = k_w4_rows<T, R, O, kAhead<T, R, O, kStaged, G>, kStaged, G>;
template <typename T, int R, int O, bool kStaged, int G>
hipError_t rows_as(const W4Args& a, hipStream_t s) {
    const dim3 grid((a.w.out_tiles + O - 1) / O, (unsigned)((a.rows + 16 * R - 1) / (16 * R)));
    const int lds = kStaged ? std::max(kPartLds<R, O>, (int)stage_bytes(a)) : kPartLds<R, O>;
    kRowsKernel<T, R, O, kStaged, G><<<grid, 64 * kWaves, lds, s>>>(a);
    return hipGetLastError();
}
template <typename T, int R, bool kStaged, int G>
hipError_t rows_of(const W4Args& a, hipStream_t s) {
    const int o = rows_o<T, R, kStaged, G>(a);
    if constexpr (kMostO<T, R, kStaged, G> >= 4)
        if (o == 4) return rows_as<T, R, 4, kStaged, G>(a, s);
    if constexpr (kMostO<T, R, kStaged, G> >= 2)
        if (o == 2) return rows_as<T, R, 2, kStaged, G>(a, s);
    return rows_as<T, R, 1, kStaged, G>(a, s);
}
template <typename T, int R, bool kStaged, int G>
hipError_t rows_prepare() {
    const auto allow = [](const void* f, int bytes) { return hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, bytes); };
    constexpr int M = kMostO<T, R, kStaged, G>, least = kStaged ? kStageBytes : 0;
    hipError_t e = allow(reinterpret_cast<const void*>(kRowsKernel<T, R, 1, kStaged, G>), std::max(least, kPartLds<R, 1>));
    if constexpr (M >= 2)
        if (e == hipSuccess) e = allow(reinterpret_cast<const void*>(kRowsKernel<T, R, 2, kStaged, G>), std::max(least, kPartLds<R, 2>));
    if constexpr (M >= 4)
        if (e == hipSuccess) e = allow(reinterpret_cast<const void*>(kRowsKernel<T, R, 4, kStaged, G>), std::max(least, kPartLds<R, 4>));
    return e;
}

template <typename T, int H, int S, int G>
constexpr int kTileLds = std::max(2 * (2 * H * 8 * Kind<T>::kTerms * 1024 + (G < S ? S : G) * 64 * H * 16), S == 1 ? 0 : 4 * 2 * H * 16 * 64 * 4);
template <typename T, int H, int S, int G>
hipError_t tile_as(const W4Args& a, hipStream_t s) {
    const int row_blocks = (int)((a.rows + 64 * H - 1) / (64 * H)), out_blocks = (a.w.n_out + kTileOuts - 1) / kTileOuts;
    const unsigned grid = (unsigned)((out_blocks + 7) / 8 * 8) * row_blocks;
    k_w4_tile<T, H, S, G><<<grid, 256 * S, kTileLds<T, H, S, G>, s>>>(a, row_blocks, out_blocks);
    return hipGetLastError();
}

template <typename T, int G>
hipError_t w4_as(const W4Args& a, hipStream_t s) {
    if constexpr (sizeof(T) == 4) {
        if (a.rows <= 16 && stage_bytes(a) <= kStageBytes) return rows_of<T, 1, true, G>(a, s);
    }
    if (a.rows <= 16) return rows_of<T, 1, false, G>(a, s);
    if (a.rows <= 32) return rows_of<T, 2, false, G>(a, s);
    // While the workgroups of 64 rows are few, the tiles' would leave compute units idle (64 rows x 128 outputs each), and a chunk takes
    // one of those 1.3 us: 4096 x 11008, 128 rows 82 us for 110 (512 workgroups), 192 rows 123 for 110; fp32 64 rows 85 for 181
    // (256), 128 rows 167 for 180, but 15,360 x 5120, 64 rows 168 for 87 (960).
    const int o = rows_o<T, 4, false, G>(a);
    if ((a.rows + 63) / 64 * ((a.w.out_tiles + o - 1) / o) <= (sizeof(T) == 2 ? 512 : 256)) return rows_of<T, 4, false, G>(a, s);
    // Eight waves of 64 rows while two such workgroups a compute unit hold all of them; four of 128 rows beyond, which widen the codes
    // half as often: 15,360 x 5120, 256 rows (480 workgroups) 70 us for 93, 512 rows 134 for 112. In fp32 the smaller one is always
    // ahead (1,500 rows 1,058 us; four waves of 64 rows 1,307, and 128 rows do not fit LDS).
    if constexpr (sizeof(T) == 2) {
        if ((a.rows + 63) / 64 * ((a.w.n_out + kTileOuts - 1) / kTileOuts) > 512) return tile_as<T, 2, 1, G>(a, s);
    }
    return tile_as<T, 1, 2, G>(a, s);
}
template <typename T>
hipError_t w4_any(const W4Args& a, hipStream_t s) {
    return a.w.per_chunk == 1 ? w4_as<T, 1>(a, s) : a.w.per_chunk == 2 ? w4_as<T, 2>(a, s) : w4_as<T, 4>(a, s);
}

template <typename T, int G>
hipError_t prepare() {
    const auto allow = [](const void* f, int bytes) { return hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, bytes); };
    if constexpr (sizeof(T) == 4) {
        const hipError_t e = rows_prepare<T, 1, true, G>();
        if (e != hipSuccess) return e;
    }
    if constexpr (sizeof(T) == 2) {
        const hipError_t e = allow(reinterpret_cast<const void*>(k_w4_tile<T, 2, 1, G>), kTileLds<T, 2, 1, G>);
        if (e != hipSuccess) return e;
    }
    for (hipError_t e : {allow(reinterpret_cast<const void*>(k_w4_tile<T, 1, 2, G>), kTileLds<T, 1, 2, G>), rows_prepare<T, 1, false, G>(),
                         rows_prepare<T, 2, false, G>(), rows_prepare<T, 4, false, G>()})
        if (e != hipSuccess) return e;
    return hipSuccess;
}
template <typename T>
hipError_t prepare_all() {
    for (hipError_t e : {prepare<T, 1>(), prepare<T, 2>(), prepare<T, 4>()})
        if (e != hipSuccess) return e;
    return hipSuccess;
}

}  // namespace

hipError_t launch_w4_pack(const W4PackArgs& a, hipStream_t s) {
    const int64_t tiles = (int64_t)a.out_tiles * a.chunks;
    k_w4_pack<<<(unsigned)std::min<int64_t>(tiles, kPackGrid), 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_w4(const W4Args& a, int x_dtype, hipStream_t s) {
    if (x_dtype == 0) return w4_any<float>(a, s);
    if (x_dtype == 1) return w4_any<__bf16>(a, s);
    return w4_any<_Float16>(a, s);
}

hipError_t w4_prepare() {
    static std::atomic<uint64_t> done{0};  // a bit per device
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
    for (hipError_t x : {prepare_all<float>(), prepare_all<__bf16>(), prepare_all<_Float16>()})
        if (x != hipSuccess) e = x;
    if (e == hipSuccess && dev < 64) done.fetch_or(1ull << dev);
    return e;
}

}  // namespace np
