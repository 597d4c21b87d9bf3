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
template <typename T, int R, int U, bool kStaged>
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
    const int64_t first_group = (int64_t)tile * w.chunks * w.per_chunk;
    const int fold = w.per_chunk == 1 ? 8 : w.per_chunk == 2 ? 10 : 15;  // products after which a group ends
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
        uint32_t scale[4], zero[4];
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
        for (int g = 0; g < 4; ++g) {
            if (g >= w.per_chunk) continue;
            const int64_t at = (first_group + c * w.per_chunk + g) * kW4Outs + col;
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
            if (fold >> s & 1) {
                const int g = w.per_chunk == 1 ? 0 : w.per_chunk == 2 ? s >> 1 : s;
                const float sc = scale_value(g == 0 ? p.scale[0] : g == 1 ? p.scale[1] : g == 2 ? p.scale[2] : p.scale[3], w.scale_dtype);
                const float z = (float)(g == 0 ? p.zero[0] : g == 1 ? p.zero[1] : g == 2 ? p.zero[2] : p.zero[3]);
#pragma unroll
                for (int r = 0; r < R; ++r) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) tot[r][j] = __builtin_fmaf(sc, __builtin_fmaf(-z, sum[r][j], part[r][j]), tot[r][j]);
                    part[r] = sum[r] = f32x4{0, 0, 0, 0};
                }
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
                const int g = w.per_chunk == 1 ? 0 : w.per_chunk == 2 ? s >> 1 : s;
                const float sc = scale_value(g == 0 ? p.scale[0] : g == 1 ? p.scale[1] : g == 2 ? p.scale[2] : p.scale[3], w.scale_dtype);
                const E8 cw = weights_of<E>(p.code[s], (int)(g == 0 ? p.zero[0] : g == 1 ? p.zero[1] : g == 2 ? p.zero[2] : p.zero[3]));
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

// Many rows: one workgroup of four waves per (16 RT rows, 128 outputs), two by two; a wave has 8 RT rows x 64 outputs. The
// workgroup's x of a chunk of 128 inputs is in LDS as operands (two chunks: one is read while the next one's loads are
// on their way), each wave widens the codes of its outputs itself.
template <typename T, int RT>
__global__ __launch_bounds__(256, 2) void k_w4_tile(W4Args a, int row_blocks, int out_blocks) {
    typedef Kind<T> Kd;
    typedef typename Kd::E E;
    typedef typename Vec8<E>::t E8;
    constexpr int N = Kd::kTerms, H = RT / 2;
    const W4View& w = a.w;
    // Workgroups go to the 8 dies in turn: a die takes its own outputs, with all rows one after the other.
    const int die = blockIdx.x & 7, nth = blockIdx.x >> 3;
    const int ob = die + 8 * (nth / row_blocks), rb = nth % row_blocks;
    if (ob >= out_blocks) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int64_t r0 = (int64_t)rb * 16 * RT;
    const int rows = (int)min((int64_t)16 * RT, a.rows - r0);
    const int half = wave & 1, tile0 = ob * 8 + (wave >> 1) * 4;
    const int fold = w.per_chunk == 1 ? 8 : w.per_chunk == 2 ? 10 : 15;
    extern __shared__ __attribute__((aligned(128))) uint8_t s_dyn[];
    E8* const s_x = reinterpret_cast<E8*>(s_dyn);  // [2][RT][4][N][64 lanes]

    // The wave stages RT of the 4 RT (row tile, product) operands.
    XRaw<T> stage[RT];
    const auto ask_x = [&](int c) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int f = wave * RT + i, rt = f >> 2, s = f & 3;
            const int k = c * kW4Ins + s * 32 + quad * 8;
            stage[i] = load_x<T>(static_cast<const T*>(a.x) + (r0 + min(16 * rt + col, rows - 1)) * a.x_row + k, k < w.n_in);
        }
    };
    const auto put_x = [&](int c) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            E8 o[N];
            operands<T>(o, stage[i]);
#pragma unroll
            for (int n = 0; n < N; ++n) s_x[(((c & 1) * RT * 4 + wave * RT + i) * N + n) * 64 + lane] = o[n];
        }
    };
    const uint8_t* tiles[4];
    int64_t groups[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int64_t tile = min(tile0 + t, w.out_tiles - 1);  // past the last: not stored
        tiles[t] = w.tiles + tile * w.chunks * kW4TileBytes + lane * 16;
        groups[t] = tile * w.chunks * w.per_chunk;
    }
    u32x4 code[4], next[4];
    const auto ask_codes = [&](u32x4* o, int c) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 4; ++t) o[t] = *reinterpret_cast<const u32x4*>(tiles[t] + (int64_t)c * kW4TileBytes);
    };
    f32x4 tot[H][4];
#pragma unroll
    for (int r = 0; r < H; ++r)
#pragma unroll
        for (int t = 0; t < 4; ++t) tot[r][t] = f32x4{0, 0, 0, 0};

    ask_x(0);
    ask_codes(code, 0);
    put_x(0);
    for (int c = 0; c < w.chunks; ++c) {
        __syncthreads();
        if (c + 1 < w.chunks) {
            ask_x(c + 1);
            ask_codes(next, c + 1);
        }
        f32x4 part[H][4], sum[H];
#pragma unroll
        for (int r = 0; r < H; ++r) {
            sum[r] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int t = 0; t < 4; ++t) part[r][t] = f32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            E8 cw[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) cw[t] = codes_of<E>(code[t][s]);
#pragma unroll
            for (int r = 0; r < H; ++r)
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const E8 x = s_x[(((c & 1) * RT * 4 + (half * H + r) * 4 + s) * N + n) * 64 + lane];
                    sum[r] = mfma(x, ones<E>(), sum[r]);
#pragma unroll
                    for (int t = 0; t < 4; ++t) part[r][t] = mfma(x, cw[t], part[r][t]);
                }
            if (fold >> s & 1) {
                const int g = w.per_chunk == 1 ? 0 : w.per_chunk == 2 ? s >> 1 : s;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int64_t at = (groups[t] + c * w.per_chunk + g) * kW4Outs + col;
                    const float sc = scale_value(load_scale(w, at), w.scale_dtype), z = w.zeros ? (float)w.zeros[at] : 8.0f;
#pragma unroll
                    for (int r = 0; r < H; ++r) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) tot[r][t][j] = __builtin_fmaf(sc, __builtin_fmaf(-z, sum[r][j], part[r][t][j]), tot[r][t][j]);
                        part[r][t] = f32x4{0, 0, 0, 0};
                    }
                }
#pragma unroll
                for (int r = 0; r < H; ++r) sum[r] = f32x4{0, 0, 0, 0};
            }
        }
        if (c + 1 < w.chunks) {
            put_x(c + 1);
#pragma unroll
            for (int t = 0; t < 4; ++t) code[t] = next[t];
        }
    }
    bool odd = false;
#pragma unroll
    for (int r = 0; r < H; ++r)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) odd |= not_finite(tot[r][t][j]);
    if (__any(odd)) {
        // Every output tile of the wave again, one row tile at a time, x from memory.
#pragma unroll 1
        for (int r = 0; r < H; ++r) {
#pragma unroll 1
            for (int t = 0; t < 4; ++t) {
                const T* const x0 = static_cast<const T*>(a.x) + (r0 + min(16 * (half * H + r) + col, rows - 1)) * a.x_row + quad * 8;
                const int64_t tile = min(tile0 + t, w.out_tiles - 1);
                f32x4 again = {0, 0, 0, 0};
#pragma unroll 1
                for (int c = 0; c < w.chunks; ++c) {
                    const u32x4 cd = *reinterpret_cast<const u32x4*>(w.tiles + (tile * w.chunks + c) * kW4TileBytes + lane * 16);
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int g = w.per_chunk == 1 ? 0 : w.per_chunk == 2 ? s >> 1 : s, k = c * kW4Ins + s * 32;
                        const int64_t at = ((tile * w.chunks + c) * w.per_chunk + g) * kW4Outs + col;
                        const float sc = scale_value(load_scale(w, at), w.scale_dtype);
                        const E8 cw = weights_of<E>(cd[s], w.zeros ? w.zeros[at] : 8);
                        E8 x[N];
                        operands_of_any<T>(x, load_x<T>(x0 + k, k + quad * 8 < w.n_in));
                        f32x4 part = {0, 0, 0, 0};
#pragma unroll
                        for (int n = 0; n < N; ++n) part = mfma(x[n], cw, part);
#pragma unroll
                        for (int j = 0; j < 4; ++j) again[j] = __builtin_fmaf(sc, part[j], again[j]);
                    }
                }
#pragma unroll
                for (int rr = 0; rr < H; ++rr)
#pragma unroll
                    for (int tt = 0; tt < 4; ++tt)
                        if (rr == r && tt == t)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (not_finite(tot[rr][tt][j])) tot[rr][tt][j] = again[j];
            }
        }
    }
#pragma unroll
    for (int r = 0; r < H; ++r)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = 16 * (half * H + r) + 4 * quad + j, out = (tile0 + t) * kW4Outs + col;
                if (row < rows && tile0 + t < w.out_tiles && out < w.n_out) put(a, r0 + row, out, tot[r][t][j]);
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

template <typename T, int R, int U>
hipError_t rows_as(const W4Args& a, hipStream_t s) {
    const dim3 grid(a.w.out_tiles, (unsigned)((a.rows + 16 * R - 1) / (16 * R)));
    k_w4_rows<T, R, U, false><<<grid, 64 * kWaves, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
constexpr int kTileRows = sizeof(T) == 2 ? 8 : 4;  // row tiles of a workgroup: what two chunks of LDS hold
template <typename T>
constexpr int kTileLds = 2 * kTileRows<T> * 4 * Kind<T>::kTerms * 1024;

template <typename T>
hipError_t w4_as(const W4Args& a, hipStream_t s) {
    if constexpr (sizeof(T) == 4) {
        if (a.rows <= 16 && stage_bytes(a) <= kStageBytes) {
            k_w4_rows<T, 1, 4, true><<<dim3(a.w.out_tiles, 1), 64 * kWaves, stage_bytes(a), s>>>(a);
            return hipGetLastError();
        }
    }
    if (a.rows <= 16) return rows_as<T, 1, sizeof(T) == 2 ? 4 : 2>(a, s);
    if (a.rows <= 32) return rows_as<T, 2, sizeof(T) == 2 ? 2 : 1>(a, s);
    if (a.rows <= 64) return rows_as<T, 4, sizeof(T) == 2 ? 2 : 1>(a, s);
    constexpr int RT = kTileRows<T>;
    const int row_blocks = (int)((a.rows + 16 * RT - 1) / (16 * RT)), out_blocks = (a.w.out_tiles + 7) / 8;
    const unsigned grid = (unsigned)((out_blocks + 7) / 8 * 8) * row_blocks;
    k_w4_tile<T, RT><<<grid, 256, kTileLds<T>, s>>>(a, row_blocks, out_blocks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_w4_pack(const W4PackArgs& a, hipStream_t s) {
    const int64_t tiles = (int64_t)a.out_tiles * a.chunks;
    k_w4_pack<<<(unsigned)std::min<int64_t>(tiles, kPackGrid), 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_w4(const W4Args& a, int x_dtype, hipStream_t s) {
    if (x_dtype == 0) return w4_as<float>(a, s);
    if (x_dtype == 1) return w4_as<__bf16>(a, s);
    return w4_as<_Float16>(a, s);
}

hipError_t w4_prepare() {
    static std::atomic<uint64_t> done{0};  // a bit per device
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
    const auto allow = [&](const void* f, int bytes) {
        const hipError_t x = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (x != hipSuccess) e = x;
    };
    allow(reinterpret_cast<const void*>(k_w4_rows<float, 1, 4, true>), kStageBytes);
    allow(reinterpret_cast<const void*>(k_w4_tile<float, kTileRows<float>>), kTileLds<float>);
    allow(reinterpret_cast<const void*>(k_w4_tile<__bf16, kTileRows<__bf16>>), kTileLds<__bf16>);
    allow(reinterpret_cast<const void*>(k_w4_tile<_Float16, kTileRows<_Float16>>), kTileLds<_Float16>);
    if (e == hipSuccess && dev < 64) done.fetch_or(1ull << dev);
    return e;
}

}  // namespace np
