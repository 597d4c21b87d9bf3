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

__device__ inline float scale_value(uint32_t raw, int dtype) {
    if (dtype == 0) return __uint_as_float(raw);
    if (dtype == 1) return __uint_as_float(raw << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)raw);
}
__device__ inline uint32_t load_scale(const W4View& w, int64_t at) {
    return w.scale_dtype == 0 ? static_cast<const uint32_t*>(w.scales)[at] : static_cast<const uint16_t*>(w.scales)[at];
}

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
constexpr int kPartStride = kW4Outs + 1;

// Few rows: one workgroup per 16 outputs and 16 R rows; its waves take every kWaves-th chunk of 128 inputs and are joined
// in LDS, in their order. A lane's 16 bytes of a tile are its operands of four products, x the other one: D row = row of x,
// D column = output. x comes from the caches (kStaged: fp32, split once per workgroup into LDS).
template <typename T, int R, int U, bool kStaged, int G>
__global__ __launch_bounds__(64 * kWaves) void k_w4_rows(W4Args a) {
    typedef Kind<T> Kd;
    typedef typename Kd::E E;
    typedef typename Vec8<E>::t E8;
    constexpr int N = Kd::kTerms;
    const W4View& w = a.w;
    const int tile = blockIdx.x, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int64_t r0 = (int64_t)blockIdx.y * 16 * R;
    const int rows = (int)min((int64_t)16 * R, a.rows - r0);
    const uint8_t* const tiles = w.tiles + (int64_t)tile * w.chunks * kW4TileBytes + lane * 16;
    const int64_t first_group = (int64_t)tile * w.chunks * G;
    __shared__ float s_part[kWaves * 16 * R * kPartStride];
    extern __shared__ __attribute__((aligned(128))) uint8_t s_dyn[];
    E* const s_x = reinterpret_cast<E*>(s_dyn);  // [N][rows][x_len]
    const int x_len = w.chunks * kW4Ins + 8;

    // Rows past the last read the last one: what they give is not stored.
    const T* xr[R];
#pragma unroll
    for (int r = 0; r < R; ++r) xr[r] = static_cast<const T*>(a.x) + (r0 + min(16 * r + col, rows - 1)) * a.x_row + quad * 8;

    struct Part {
        u32x4 code;
        XRaw<T> x[kStaged ? 1 : R][4];
        uint32_t scale[G], zero[G];
    };
    const auto ask = [&](Part& p, int c) __attribute__((always_inline)) {
        p.code = *reinterpret_cast<const u32x4*>(tiles + (int64_t)c * kW4TileBytes);
        if constexpr (!kStaged) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int s = 0; s < 4; ++s) p.x[r][s] = load_x<T>(xr[r] + c * kW4Ins + s * 32, c * kW4Ins + s * 32 + quad * 8 < w.n_in);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int64_t at = (first_group + c * G + g) * kW4Outs + col;
            p.scale[g] = load_scale(w, at);
            p.zero[g] = w.zeros ? w.zeros[at] : 8;
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
    f32x4 tot[R];
#pragma unroll
    for (int r = 0; r < R; ++r) tot[r] = f32x4{0, 0, 0, 0};
    const auto products = [&](const Part& p, int c) __attribute__((always_inline)) {
        f32x4 part[R], sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r) part[r] = sum[r] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const E8 cw = codes_of<E>(p.code[s]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                E8 x[N];
                x_of(x, p, c, r, s);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    part[r] = mfma(x[n], cw, part[r]);
                    sum[r] = mfma(x[n], ones<E>(), sum[r]);
                }
            }
            if ((s + 1) * G % 4 == 0) {  // a group ends
                const int g = s * G / 4;
                const float sc = scale_value(p.scale[g], w.scale_dtype);
                const float z = (float)p.zero[g];
#pragma unroll
                for (int r = 0; r < R; ++r) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) tot[r][j] = __builtin_fmaf(sc, __builtin_fmaf(-z, sum[r][j], part[r][j]), tot[r][j]);
                    part[r] = sum[r] = f32x4{0, 0, 0, 0};
                }
                if (R > 1) __builtin_amdgcn_sched_barrier(0);  // as few registers as there are
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
        for (int j = 0; j < 4; ++j) odd |= not_finite(tot[r][j]);
    if (__any(odd)) {
        f32x4 again[R];
#pragma unroll
        for (int r = 0; r < R; ++r) again[r] = f32x4{0, 0, 0, 0};
#pragma unroll 1
        for (int c = wave; c < w.chunks; c += kWaves) {
            Part p;
            ask(p, c);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int g = s * G / 4;
                const float sc = scale_value(p.scale[g], w.scale_dtype);
                const E8 cw = weights_of<E>(p.code[s], (int)p.zero[g]);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    E8 x[N];
                    operands_of_any<T>(x, load_x<T>(xr[r] + c * kW4Ins + s * 32, c * kW4Ins + s * 32 + quad * 8 < w.n_in));
                    f32x4 part = {0, 0, 0, 0};
#pragma unroll
                    for (int n = 0; n < N; ++n) part = mfma(x[n], cw, part);
#pragma unroll
                    for (int j = 0; j < 4; ++j) again[r][j] = __builtin_fmaf(sc, part[j], again[r][j]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (not_finite(tot[r][j])) tot[r][j] = again[r][j];
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) s_part[(wave * 16 * R + 16 * r + 4 * quad + j) * kPartStride + col] = tot[r][j];
    __syncthreads();
    for (int i = threadIdx.x; i < rows * kW4Outs; i += 64 * kWaves) {
        const int r = i / kW4Outs, o = i & (kW4Outs - 1);
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) v += s_part[(k * 16 * R + r) * kPartStride + o];
        if (tile * kW4Outs + o < w.n_out) put(a, r0 + r, tile * kW4Outs + o, v);
    }
}

// Many rows: one workgroup of four waves per (64 H rows, 128 outputs), two by two; a wave has 32 H rows x 64 outputs, in products
// of 32x32x16. The workgroup's x of a chunk of 128 inputs is in LDS as operands (two chunks: one is read while the next one's
// loads are on their way), with the sums of each row and group, three bf16 terms of them, that take the zero points out: one
// more product per group, with -z as the other operand. Each wave widens the codes of its outputs itself.
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

template <typename T, int H, int G>
__global__ __launch_bounds__(256, 2) void k_w4_tile(W4Args a, int row_blocks, int out_blocks) {
    typedef Kind<T> Kd;
    typedef typename Kd::E E;
    typedef typename Vec8<E>::t E8;
    constexpr int N = Kd::kTerms, kRows = 64 * H;
    const W4View& w = a.w;
    // Workgroups go to the 8 dies in turn: a die takes its own outputs, with all rows one after the other.
    const int die = blockIdx.x & 7, nth = blockIdx.x >> 3;
    const int ob = die + 8 * (nth / row_blocks), rb = nth % row_blocks;
    if (ob >= out_blocks) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int64_t r0 = (int64_t)rb * kRows;
    const int rows = (int)min((int64_t)kRows, a.rows - r0);
    const int row0 = (wave & 1) * 32 * H, tile0 = ob * 8 + (wave >> 1) * 4;
    extern __shared__ __attribute__((aligned(128))) uint8_t s_dyn[];
    E8* const s_x = reinterpret_cast<E8*>(s_dyn);  // [2][2 H row tiles][8 steps][N][2 halves][32 rows, changed places]
    constexpr int kBuf = 2 * H * 8 * N * 64;
    bf16x8* const s_sum = reinterpret_cast<bf16x8*>(s_dyn + 2 * kBuf * 16);  // [2][G][rows]

    // Staging: a wave brings 16 H rows in units of 16 rows x 32 inputs: lane 4 r + q has quad q of row r. Places in LDS: row r of (step,
    // half) at r ^ 4 q, so that a unit's 64 stores meet no bank twice.
    XRaw<T> stage[H][4];
    const int sr = lane >> 2, sq = lane & 3;
    const T* xs[H];
#pragma unroll
    for (int u = 0; u < H; ++u) xs[u] = static_cast<const T*>(a.x) + (r0 + min(wave * 16 * H + u * 16 + sr, rows - 1)) * a.x_row + sq * 8;
    const auto ask_x = [&](int c) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < H; ++u)
#pragma unroll
            for (int s = 0; s < 4; ++s) stage[u][s] = load_x<T>(xs[u] + c * kW4Ins + s * 32, c * kW4Ins + s * 32 + sq * 8 < w.n_in);
    };
    const auto put_x = [&](int c) __attribute__((always_inline)) {
        E8* const to = s_x + (c & 1) * kBuf;
        bf16x8* const sums = s_sum + (c & 1) * G * kRows;
#pragma unroll
        for (int u = 0; u < H; ++u) {
            const int row = wave * 16 * H + u * 16 + sr;
            float part[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                E8 o[N];
                operands<T>(o, stage[u][s]);
#pragma unroll
                for (int n = 0; n < N; ++n)
                    to[((((row >> 5) * 8 + 2 * s + (sq >> 1)) * N + n) * 2 + (sq & 1)) * 32 + ((row & 31) ^ (4 * sq))] = o[n];
                part[s] = quad_sum(sum8<T>(stage[u][s]));
            }
            // Lane q writes group q's sum.
            float v = G == 4 ? (sq == 0 ? part[0] : sq == 1 ? part[1] : sq == 2 ? part[2] : part[3])
                             : G == 2 ? (sq ? part[2] + part[3] : part[0] + part[1]) : (part[0] + part[1]) + (part[2] + part[3]);
            u32x4 t = {0, 0, 0, 0};
            const uint32_t t0 = __float_as_uint(v) & 0xffff0000u;
            v -= __uint_as_float(t0);
            const uint32_t t1 = __float_as_uint(v) & 0xffff0000u;
            v -= __uint_as_float(t1);
            t[0] = t0 >> 16 | t1;
            t[1] = __float_as_uint(v) >> 16;
            if (sq < G) sums[sq * kRows + row] = __builtin_bit_cast(bf16x8, t);
        }
    };
    // Codes of outputs 32 t + col: quads h and h + 2 of the tile.
    const uint8_t* tiles[2];
    int64_t groups[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int64_t tile = min(tile0 + 2 * t + (col >> 4), w.out_tiles - 1);  // past the last: not stored
        tiles[t] = w.tiles + tile * w.chunks * kW4TileBytes + (h * 16 + (col & 15)) * 16;
        groups[t] = tile * w.chunks * G * kW4Outs + (col & 15);
    }
    u32x4 code[2][2], next[2][2];
    uint32_t scale[2][G], zero[2][G], next_scale[2][G], next_zero[2][G];
    const auto ask_codes = [&](u32x4 (&o)[2][2], uint32_t (&sc)[2][G], uint32_t (&z)[2][G], int c) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int e = 0; e < 2; ++e) o[t][e] = *reinterpret_cast<const u32x4*>(tiles[t] + (int64_t)c * kW4TileBytes + e * 512);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int64_t at = groups[t] + (c * G + g) * kW4Outs;
                sc[t][g] = load_scale(w, at);
                z[t][g] = w.zeros ? w.zeros[at] : 8;
            }
        }
    };
    f32x16 tot[H][2];
#pragma unroll
    for (int r = 0; r < H; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) tot[r][t][j] = 0.0f;

    ask_x(0);
    ask_codes(code, scale, zero, 0);
    put_x(0);
    for (int c = 0; c < w.chunks; ++c) {
        __syncthreads();
        if (c + 1 < w.chunks) {
            ask_x(c + 1);
            ask_codes(next, next_scale, next_zero, c + 1);
        }
        const E8* const from = s_x + (c & 1) * kBuf + (row0 >> 5) * 8 * N * 64 + h * 32;
        const bf16x8* const sums = s_sum + (c & 1) * G * kRows + row0 + col;
        f32x16 part[H][2];
#pragma unroll
        for (int r = 0; r < H; ++r)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < 16; ++j) part[r][t][j] = 0.0f;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                E8 cw[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) cw[t] = codes_of<E>(code[t][e][s]);
#pragma unroll
                for (int r = 0; r < H; ++r)
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const E8 x = from[((r * 8 + 2 * s + e) * N + n) * 64 + (col ^ (4 * (h + 2 * e)))];
#pragma unroll
                        for (int t = 0; t < 2; ++t) part[r][t] = mfma(x, cw[t], part[r][t]);
                    }
            }
            if ((s + 1) * G % 4 == 0) {  // a group ends
                const int g = s * G / 4;
                bf16x8 xs8[H];
#pragma unroll
                for (int r = 0; r < H; ++r) xs8[r] = sums[g * kRows + 32 * r];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float sc = scale_value(scale[t][g], w.scale_dtype);
                    const float z = (float)zero[t][g];
                    const uint32_t zb = h ? 0u : __float_as_uint(-z);  // whole numbers up to 15: the upper half is bf16
                    const bf16x8 minus = __builtin_bit_cast(bf16x8, u32x4{zb >> 16 | zb, zb >> 16, 0, 0});
#pragma unroll
                    for (int r = 0; r < H; ++r) {
                        part[r][t] = mfma(xs8[r], minus, part[r][t]);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            tot[r][t][j] = __builtin_fmaf(sc, part[r][t][j], tot[r][t][j]);
                            part[r][t][j] = 0.0f;
                        }
                    }
                }
                if (G > 1) __builtin_amdgcn_sched_barrier(0);  // two groups' sums at a time would not fit
            }
        }
        if (c + 1 < w.chunks) {
            put_x(c + 1);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int e = 0; e < 2; ++e) code[t][e] = next[t][e];
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    scale[t][g] = next_scale[t][g];
                    zero[t][g] = next_zero[t][g];
                }
            }
        }
    }
    bool odd = false;
#pragma unroll
    for (int r = 0; r < H; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) odd |= not_finite(tot[r][t][j]);
    if (__any(odd)) {
        // The wave's products again, one at a time, x from memory.
#pragma unroll 1
        for (int r = 0; r < H; ++r) {
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
                const T* const x0 = static_cast<const T*>(a.x) + (r0 + min(row0 + 32 * r + col, rows - 1)) * a.x_row;
                const int64_t tile = min(tile0 + 2 * t + (col >> 4), w.out_tiles - 1);
                f32x16 again;
#pragma unroll
                for (int j = 0; j < 16; ++j) again[j] = 0.0f;
#pragma unroll 1
                for (int c = 0; c < w.chunks; ++c) {
#pragma unroll 1
                    for (int e = 0; e < 2; ++e) {
                        const int q = h + 2 * e;
                        const u32x4 cd = *reinterpret_cast<const u32x4*>(w.tiles + (tile * w.chunks + c) * kW4TileBytes + (q * 16 + (col & 15)) * 16);
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const int g = s * G / 4, k = c * kW4Ins + s * 32 + q * 8;
                            const int64_t at = ((tile * w.chunks + c) * G + g) * kW4Outs + (col & 15);
                            const float sc = scale_value(load_scale(w, at), w.scale_dtype);
                            const E8 cw = weights_of<E>(cd[s], w.zeros ? w.zeros[at] : 8);
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
                for (int rr = 0; rr < H; ++rr)
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt)
                        if (rr == r && tt == t)
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (not_finite(tot[rr][tt][j])) tot[rr][tt][j] = again[j];
            }
        }
    }
#pragma unroll
    for (int r = 0; r < H; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int row = row0 + 32 * r + 8 * (j >> 2) + 4 * h + (j & 3), tile = tile0 + 2 * t + (col >> 4), out = tile * kW4Outs + (col & 15);
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
        if (a.scale_bytes == 4) static_cast<uint32_t*>(a.scales_out)[i] = in ? static_cast<const uint32_t*>(a.scales)[from] : 0;
        else static_cast<uint16_t*>(a.scales_out)[i] = in ? static_cast<const uint16_t*>(a.scales)[from] : 0;
        if (a.zeros) a.zeros_out[i] = in ? a.zeros[from] & 15 : 0;
    }
}

// LDS for x of one workgroup of k_w4_rows, split (fp32); at most this much of it is used.
constexpr int kStageBytes = 96 * 1024;
int stage_bytes(const W4Args& a) { return (int)std::min<int64_t>(1 << 30, a.rows * (a.w.chunks * kW4Ins + 8) * 3 * 2); }

template <typename T, int R, int U, int G>
hipError_t rows_as(const W4Args& a, hipStream_t s) {
    const dim3 grid(a.w.out_tiles, (unsigned)((a.rows + 16 * R - 1) / (16 * R)));
    k_w4_rows<T, R, U, false, G><<<grid, 64 * kWaves, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
constexpr int kTileH = sizeof(T) == 2 ? 2 : 1;  // what two chunks of LDS hold
template <typename T, int G>
constexpr int kTileLds = 2 * (2 * kTileH<T> * 8 * Kind<T>::kTerms * 1024 + G * 64 * kTileH<T> * 16);

template <typename T, int G>
hipError_t w4_as(const W4Args& a, hipStream_t s) {
    if constexpr (sizeof(T) == 4) {
        if (a.rows <= 16 && stage_bytes(a) <= kStageBytes) {
            k_w4_rows<T, 1, 4, true, G><<<dim3(a.w.out_tiles, 1), 64 * kWaves, stage_bytes(a), s>>>(a);
            return hipGetLastError();
        }
    }
    if (a.rows <= 16) return rows_as<T, 1, sizeof(T) == 2 ? 4 : 2, G>(a, s);
    if (a.rows <= 32) return rows_as<T, 2, sizeof(T) == 2 ? 2 : 1, G>(a, s);
    if (a.rows <= 64) return rows_as<T, 4, sizeof(T) == 2 ? 2 : 1, G>(a, s);
    constexpr int H = kTileH<T>;
    const int row_blocks = (int)((a.rows + 64 * H - 1) / (64 * H)), out_blocks = (a.w.n_out + kTileOuts - 1) / kTileOuts;
    const unsigned grid = (unsigned)((out_blocks + 7) / 8 * 8) * row_blocks;
    k_w4_tile<T, H, G><<<grid, 256, kTileLds<T, G>, s>>>(a, row_blocks, out_blocks);
    return hipGetLastError();
}
template <typename T>
hipError_t w4_any(const W4Args& a, hipStream_t s) {
    return a.w.per_chunk == 1 ? w4_as<T, 1>(a, s) : a.w.per_chunk == 2 ? w4_as<T, 2>(a, s) : w4_as<T, 4>(a, s);
}

template <typename T, int G>
hipError_t prepare() {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_w4_tile<T, kTileH<T>, G>), hipFuncAttributeMaxDynamicSharedMemorySize, kTileLds<T, G>);
    if constexpr (sizeof(T) == 4) {
        if (e == hipSuccess)
            e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_w4_rows<T, 1, 4, true, G>), hipFuncAttributeMaxDynamicSharedMemorySize, kStageBytes);
    }
    return e;
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
