// Host side of the rotary positions (np_rope_* of include/np.h): the pairs' turns, the checks of every call, and the
// launches. Nothing is enqueued before every check of a call has passed.
#include <hip/hip_runtime.h>

#include <cmath>
#include <vector>

#include "kv_host.hpp"
#include "rope_internal.hpp"

using namespace np;

struct np_rope {
    np_rope_desc desc{};
    uint64_t* turns = nullptr;  // device, [rot_dim / 2]
    ~np_rope() {
        if (turns) (void)hipFree(turns);
    }
};

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;
// What a pair may turn by per position, in radians: of more, turn_bits() would lose bits behind the point.
constexpr double kMostTurn = 1099511627776.0;
// Enough waves to fill the device: below, a row's heads go to several waves (each works out the angles again).
constexpr int64_t kFullWaves = 256 * 16;
// A launch has at most 2^32 - 1 threads along x, np_rope_apply's in workgroups of 256.
constexpr int64_t kMaxGroups = (int64_t)1 << 24;

// What pair i turns by per position, in radians.
double freq_of(const np_rope_desc& D, int i) {
    if (D.freqs) return D.freqs[i];
    const double rot = D.rot_dim;
    const double base = D.scaling == NP_ROPE_NTK ? D.base * std::pow(D.factor, rot / (rot - 2)) : D.base;
    const double f = std::pow(base, -2.0 * i / rot);
    if (D.scaling == NP_ROPE_LINEAR) return f / D.factor;
    if (D.scaling != NP_ROPE_BLEND) return f;
    const double keep = std::fmin(1.0, std::fmax(0.0, (D.context * f / kTwoPi - D.low) / (D.high - D.low)));
    return f * keep + f / D.factor * (1.0 - keep);
}

np_status check_desc(const np_rope_desc& D) {
    if (D.head_dim < 8 || D.head_dim > kMaxHeadDim || D.head_dim % 8)
        return fail(NP_EINVAL, "head_dim=%d must be a multiple of 8 in [8, %d]", D.head_dim, kMaxHeadDim);
    if (D.rot_dim < 0 || D.rot_dim > D.head_dim || D.rot_dim % 2)
        return fail(NP_EINVAL, "rot_dim=%d must be even, in [0, head_dim=%d]", D.rot_dim, D.head_dim);
    if (D.layout != NP_ROPE_HALF && D.layout != NP_ROPE_INTERLEAVED) return fail(NP_EINVAL, "unknown layout %d", D.layout);
    if (!(std::isfinite(D.amplitude) && D.amplitude > 0.0f)) return fail(NP_EINVAL, "amplitude=%g must be positive and finite", D.amplitude);
    if (D.freqs) {
        for (int i = 0; i < D.rot_dim / 2; ++i)
            if (!(std::fabs(D.freqs[i]) <= kMostTurn)) return fail(NP_EINVAL, "freqs[%d]=%g must be at most 2^40", i, D.freqs[i]);
        return NP_OK;
    }
    if (!(std::isfinite(D.base) && D.base > 0.0)) return fail(NP_EINVAL, "base=%g must be positive and finite", D.base);
    if (D.scaling < NP_ROPE_PLAIN || D.scaling > NP_ROPE_BLEND) return fail(NP_EINVAL, "unknown scaling %d", D.scaling);
    if (D.scaling != NP_ROPE_PLAIN && !(std::isfinite(D.factor) && D.factor > 0.0))
        return fail(NP_EINVAL, "factor=%g must be positive and finite", D.factor);
    if (D.scaling == NP_ROPE_NTK && D.rot_dim == 2) return fail(NP_EINVAL, "a larger base does not change the only pair of rot_dim=2");
    if (D.scaling == NP_ROPE_BLEND && !(D.context > 0 && std::isfinite(D.low) && std::isfinite(D.high) && D.low < D.high))
        return fail(NP_EINVAL, "context=%lld must be positive and low=%g below high=%g", (long long)D.context, D.low, D.high);
    for (int i = 0; i < D.rot_dim / 2; ++i)
        if (!(std::fabs(freq_of(D, i)) <= kMostTurn)) return fail(NP_EINVAL, "pair %d turns by %g a position: more than 2^40", i, freq_of(D, i));
    return NP_OK;
}

// 1 / (2 pi): its first 64 bits, and 64 of what they leave out.
constexpr long double kTurns = 0xa2f9836e4e44152ap-66L, kTurnsRest = -0xf62a0b82b2c88fc9p-136L;
// f radians as a fraction of a turn, to the nearest 2^-64 (whole turns do not count), for |f| <= kMostTurn.
uint64_t turn_bits(double f) {
    const long double a = std::fabs(f), t = a * kTurns, rest = std::fma(a, kTurns, -t) + a * kTurnsRest;  // t + rest turns
    const long double part = (t - std::floor(t)) * 18446744073709551616.0L, whole = std::floor(part);
    const uint64_t bits = (uint64_t)whole + (uint64_t)std::llround(part - whole + rest * 18446744073709551616.0L);
    return f < 0.0 ? 0 - bits : bits;
}

np_status create(const np_rope_desc* desc, np_rope** out) {
    if (!desc || !out) return fail(NP_EINVAL, "desc and out must not be NULL");
    *out = nullptr;
    const np_rope_desc& D = *desc;
    const np_status st = check_desc(D);
    if (st != NP_OK) return st;
    struct Holder {
        np_rope* r = new np_rope();
        ~Holder() { delete r; }
    } hold;
    std::vector<uint64_t> bits(std::max(1, D.rot_dim / 2), 0);
    for (int i = 0; i < D.rot_dim / 2; ++i) bits[i] = turn_bits(freq_of(D, i));
    int ndev = 0;
    NP_HIP(hipGetDeviceCount(&ndev));
    if (D.device < 0 || D.device >= ndev) return fail(NP_EINVAL, "device %d out of range [0, %d)", D.device, ndev);
    DeviceGuard g(D.device);
    if (!g.ok) return fail(NP_EHIP, "hipSetDevice(%d) failed", D.device);
    hold.r->desc = D;
    hold.r->desc.freqs = nullptr;  // read, not kept
    if (hipMalloc((void**)&hold.r->turns, bits.size() * sizeof(uint64_t)) != hipSuccess) {
        (void)hipGetLastError();
        return fail(NP_ENOMEM, "cannot allocate %zu bytes", bits.size() * sizeof(uint64_t));
    }
    NP_HIP(hipMemcpy(hold.r->turns, bits.data(), bits.size() * sizeof(uint64_t), hipMemcpyHostToDevice));
    *out = hold.r;
    hold.r = nullptr;
    return NP_OK;
}

RopeView view(const np_rope* r, float eps) {
    RopeView v;
    v.turns = r->turns;
    v.amplitude = r->desc.amplitude;
    v.eps = eps;
    v.hd = r->desc.head_dim;
    v.rot = r->desc.rot_dim;
    v.layout = r->desc.layout;
    return v;
}

np_status check_call(const np_rope* r, int32_t dtype, float eps) {
    if (!r) return fail(NP_EINVAL, "rope must not be NULL");
    if (dtype != NP_F32 && dtype != NP_BF16 && dtype != NP_F16) return fail(NP_EINVAL, "unknown dtype %d", dtype);
    if (!(std::isfinite(eps) && eps >= 0.0f)) return fail(NP_EINVAL, "eps=%g must be finite and not negative", eps);
    return NP_OK;
}

// Without rows a tensor may have no address.
const void* address(const void* p, int64_t rows) { return p || rows > 0 ? p : reinterpret_cast<const void*>(16); }

// The heads of `rows` rows: addresses, strides, and that the results do not overlap each other.
np_status check_tensor(const np_rope* r, int64_t rows, int32_t heads, const void* in, const void* out, const float* weight, const int64_t* S,
                       int32_t dtype, const char* what) {
    const int hd = r->desc.head_dim, dev = r->desc.device;
    np_status st;
    if ((st = check_rows(nullptr, address(in, rows), S[0], S[1], dtype, what)) != NP_OK) return st;
    if ((st = check_rows(nullptr, address(out, rows), S[2], S[3], dtype, "the result")) != NP_OK) return st;
    const __int128 row = S[2], head = S[3];
    if (!((head >= hd || heads == 1) && (row >= (heads - 1) * head + hd || rows <= 1)) &&
        !((row >= hd || rows <= 1) && (head >= (rows - 1) * row + hd || heads == 1)))
        return fail(NP_EINVAL, "%s: the result's strides (%lld, %lld) make rows or heads overlap", what, (long long)S[2], (long long)S[3]);
    if (in == out && (S[0] != S[2] || S[1] != S[3]) && rows > 0)
        return fail(NP_EINVAL, "%s: in place, the result must have the input's strides", what);
    if (weight && !aligned16(weight)) return fail(NP_EINVAL, "%s: the weights must be 16-byte aligned", what);
    if (in && (st = check_io_ptr(in, dev, what, "rope")) != NP_OK) return st;
    if (out && (st = check_io_ptr(out, dev, "the result", "rope")) != NP_OK) return st;
    if (weight && (st = check_io_ptr(weight, dev, "the weights", "rope")) != NP_OK) return st;
    return NP_OK;
}

RopeTensor tensor(const void* in, void* out, const float* weight, const int64_t* S, int32_t heads) {
    RopeTensor t;
    t.in = in;
    t.out = out;
    t.weight = weight;
    t.in_row = S[0];
    t.in_head = S[1];
    t.out_row = S[2];
    t.out_head = S[3];
    t.heads = heads;
    return t;
}

// From twice as many new tokens x key heads on, a workgroup takes several heads of its page and works their angles out once; as many
// as leave 256 workgroups of 64 tokens.
constexpr int64_t kFullKeys = 256 * 64;
// Groups of heads that a wave takes one after the other: all of a row's where rows alone fill the device.
int32_t groups_per_wave(int64_t rows, int groups) {
    const int64_t shares = std::min<int64_t>(groups, (kFullWaves + rows - 1) / rows);
    return (int32_t)((groups + shares - 1) / shares);
}

np_status apply(const np_rope* r, int64_t rows, const int32_t* positions, int32_t first, const void* q, void* q_out, int32_t n_heads, const float* q_weight,
                const void* k, void* k_out, int32_t n_kv_heads, const float* k_weight, float eps, int32_t dtype, const int64_t* strides, hipStream_t s) {
    np_status st = check_call(r, dtype, eps);
    if (st != NP_OK) return st;
    const int hd = r->desc.head_dim;
    if (rows < 0 || rows > (int64_t)1 << 28) return fail(NP_EINVAL, "rows=%lld must be in [0, 2^28]", (long long)rows);
    if (n_heads < 1 || n_heads > 4096 || n_kv_heads < 0 || n_kv_heads > 4096)
        return fail(NP_EINVAL, "n_heads=%d must be in [1, 4096], n_kv_heads=%d in [0, 4096]", n_heads, n_kv_heads);
    if (!positions && rows > 0 && first > INT32_MAX - (rows - 1))
        return fail(NP_EINVAL, "positions %d .. %lld do not fit in 32 bits", first, (long long)first + rows - 1);
    if (positions && ((uintptr_t)positions & 3u)) return fail(NP_EINVAL, "positions must be 4-byte aligned");
    if (!n_kv_heads && (k || k_out || k_weight)) return fail(NP_EINVAL, "keys without heads");
    const int64_t qr = (int64_t)n_heads * hd, kr = (int64_t)n_kv_heads * hd;
    const int64_t plain[8] = {qr, hd, qr, hd, kr, hd, kr, hd};
    const int64_t* const S = strides ? strides : plain;
    if ((st = check_tensor(r, rows, n_heads, q, q_out, q_weight, S, dtype, "q")) != NP_OK) return st;
    if (n_kv_heads && (st = check_tensor(r, rows, n_kv_heads, k, k_out, k_weight, S + 4, dtype, "k")) != NP_OK) return st;
    if (positions && (st = check_io_ptr(positions, r->desc.device, "positions", "rope")) != NP_OK) return st;
    if (rows == 0) return NP_OK;
    RopeArgs a;
    a.rope = view(r, eps);
    a.x[0] = tensor(q, q_out, q_weight, S, n_heads);
    a.x[1] = tensor(k, k_out, k_weight, S + 4, n_kv_heads);
    a.positions = positions;
    a.first = first;
    a.rows = rows;
    const int groups = rope_groups(hd, n_heads + n_kv_heads);
    a.per = groups_per_wave(rows, groups);
    if (rows * ((groups + a.per - 1) / a.per) / 4 >= kMaxGroups - 1) return fail(NP_EINVAL, "%lld rows in one call are too many", (long long)rows);
    DeviceGuard g(r->desc.device);
    if (!g.ok) return fail(NP_EHIP, "hipSetDevice(%d) failed", r->desc.device);
    NP_HIP(launch_rope(a, dtype, s));
    return NP_OK;
}

np_status append(const np_rope* r, np_kv* kv, int32_t layer, const void* q, void* q_out, const void* k, const void* v, const float* q_weight,
                 const float* k_weight, float eps, int32_t dtype, const int64_t* strides, hipStream_t s) {
    np_status st = check_call(r, dtype, eps);
    if (st != NP_OK) return st;
    if ((st = check_layer_io(kv, layer, dtype)) != NP_OK) return st;
    const np_kv_desc& D = kv->desc;
    if (D.head_dim != r->desc.head_dim) return fail(NP_EINVAL, "the cache's head_dim=%d is not the rope's %d", D.head_dim, r->desc.head_dim);
    if (kv->host_only()) return fail(NP_ESTATE, "a bookkeeping-only cache holds no tokens");
    if (D.device != r->desc.device) return fail(NP_EINVAL, "the cache is on device %d, the rope on %d", D.device, r->desc.device);
    int64_t rows = 0;
    for (int32_t f : kv->b_fresh) rows += f;
    const int64_t qr = (int64_t)D.n_heads * D.head_dim, kr = (int64_t)D.n_kv_heads * D.head_dim, hd = D.head_dim;
    const int64_t plain[8] = {qr, hd, qr, hd, kr, hd, kr, hd};
    const int64_t* const S = strides ? strides : plain;
    if ((st = check_tensor(r, rows, D.n_heads, q, q_out, q_weight, S, dtype, "q")) != NP_OK) return st;
    if ((st = check_rows(kv, k, S[4], S[5], dtype, "k")) != NP_OK) return st;
    if ((st = check_rows(kv, v, S[6], S[7], dtype, "v")) != NP_OK) return st;
    if (k_weight && !aligned16(k_weight)) return fail(NP_EINVAL, "k: the weights must be 16-byte aligned");
    if ((st = check_io_ptr(k, D.device, "k", "cache")) != NP_OK) return st;
    if ((st = check_io_ptr(v, D.device, "v", "cache")) != NP_OK) return st;
    if (k_weight && (st = check_io_ptr(k_weight, D.device, "the weights", "cache")) != NP_OK) return st;
    if (rows == 0) return NP_OK;
    RopeAppendArgs a;
    a.kv = kv->view();
    a.rope = view(r, eps);
    a.q = tensor(q, q_out, q_weight, S, D.n_heads);
    a.kx[0] = k;
    a.kx[1] = v;
    a.k_weight = k_weight;
    for (int i = 0; i < 2; ++i) {
        a.row_stride[i] = S[4 + 2 * i];
        a.head_stride[i] = S[5 + 2 * i];
    }
    a.layer = layer;
    a.rows = (int32_t)rows;
    fill_batch(kv, a.b, [&](int i) {
        const int b = kv->b_before[i], f = kv->b_fresh[i];
        return f ? kv->pages_for((int64_t)b + f) - (b >> kv->page_shift) : 0;
    });
    const int groups = rope_groups(D.head_dim, D.n_heads);
    a.per = groups_per_wave(rows, groups);
    a.heads = (int32_t)std::clamp<int64_t>(rows * D.n_kv_heads / kFullKeys, 1, D.n_kv_heads);
    if (append_grid(a) * append_threads(kv->page_shift, D.head_dim, kv->slabs) >> 32)
        return fail(NP_EINVAL, "%d pages of %d heads and %lld rows in one call are too many", a.b.item0[a.b.n], D.n_kv_heads, (long long)rows);
    std::optional<DeviceGuard> g;
    if ((st = make_current(kv, g)) != NP_OK) return st;
    NP_HIP(launch_rope_append(a, dtype, s));
    return NP_OK;
}

}  // namespace

extern "C" {

np_status np_rope_freqs(const np_rope_desc* desc, double* freqs) {
    if (!desc || (!freqs && desc->rot_dim)) return fail(NP_EINVAL, "desc and freqs must not be NULL");
    const np_status st = check_desc(*desc);
    if (st != NP_OK) return st;
    for (int i = 0; i < desc->rot_dim / 2; ++i) freqs[i] = freq_of(*desc, i);
    return NP_OK;
}

np_status np_rope_create(const np_rope_desc* desc, np_rope** out) {
    return guarded([&] { return create(desc, out); });
}

np_status np_rope_destroy(np_rope* rope) {
    if (!rope) return fail(NP_EINVAL, "rope must not be NULL");
    DeviceGuard g(rope->desc.device);
    CaptureGuard c;
    delete rope;  // hipFree waits for the device
    return NP_OK;
}

np_status np_rope_apply(const np_rope* rope, int64_t rows, const int32_t* positions, int32_t first, const void* q, void* q_out, int32_t n_heads,
                        const float* q_weight, const void* k, void* k_out, int32_t n_kv_heads, const float* k_weight, float eps, int32_t dtype,
                        const int64_t* strides, void* stream) {
    return guarded([&] {
        return apply(rope, rows, positions, first, q, q_out, n_heads, q_weight, k, k_out, n_kv_heads, k_weight, eps, dtype, strides, (hipStream_t)stream);
    });
}

np_status np_rope_append(const np_rope* rope, np_kv* kv, int32_t layer, const void* q, void* q_out, const void* k, const void* v, const float* q_weight,
                         const float* k_weight, float eps, int32_t dtype, const int64_t* strides, void* stream) {
    return guarded([&] { return append(rope, kv, layer, q, q_out, k, v, q_weight, k_weight, eps, dtype, strides, (hipStream_t)stream); });
}

}  // extern "C"
