// Host side of the products with 4-bit weights (np_w4_* of include/np.h): laying out the weights once, the checks of every
// call, and the launches. Nothing is enqueued before every check of a call has passed.
#include <hip/hip_runtime.h>

#include "kv_host.hpp"
#include "w4_internal.hpp"

using namespace np;

struct np_w4 {
    np_w4_desc desc{};
    W4View view{};
    uint8_t* tiles = nullptr;
    uint32_t* scales = nullptr;
    ~np_w4() {
        if (tiles) (void)hipFree(tiles);
        if (scales) (void)hipFree(scales);
    }
};

namespace {

bool known(int32_t dtype) { return dtype == NP_F32 || dtype == NP_BF16 || dtype == NP_F16; }

np_status create(const np_w4_desc* desc, np_w4** out) {
    if (!desc || !out) return fail(NP_EINVAL, "desc and out must not be NULL");
    *out = nullptr;
    const np_w4_desc& D = *desc;
    if (D.n_out < 1 || D.n_out > 1 << 20) return fail(NP_EINVAL, "n_out=%d must be in [1, 2^20]", D.n_out);
    if (D.n_in < 8 || D.n_in > 1 << 17 || D.n_in % 8) return fail(NP_EINVAL, "n_in=%d must be a multiple of 8 in [8, 2^17]", D.n_in);
    if (D.group != 32 && D.group != 64 && (D.group < kW4Ins || D.group % kW4Ins || D.group > 1 << 17))
        return fail(NP_EINVAL, "group=%d must be 32, 64 or a multiple of 128 up to 2^17", D.group);
    if (!known(D.scale_dtype)) return fail(NP_EINVAL, "unknown scale_dtype %d", D.scale_dtype);
    const int sb = elem_bytes(D.scale_dtype);
    if (!D.codes || ((uintptr_t)D.codes & 3u)) return fail(NP_EINVAL, "codes must be a 4-byte aligned device pointer");
    if (!D.scales || (uintptr_t)D.scales % sb) return fail(NP_EINVAL, "scales must be a device pointer, aligned to its type");
    int ndev = 0;
    NP_HIP(hipGetDeviceCount(&ndev));
    if (D.device < 0 || D.device >= ndev) return fail(NP_EINVAL, "device %d out of range [0, %d)", D.device, ndev);
    DeviceGuard g(D.device);
    if (!g.ok) return fail(NP_EHIP, "hipSetDevice(%d) failed", D.device);
    np_status st;
    if ((st = check_io_ptr(D.codes, D.device, "codes", "weights")) != NP_OK) return st;
    if ((st = check_io_ptr(D.scales, D.device, "scales", "weights")) != NP_OK) return st;
    if (D.zeros && (st = check_io_ptr(D.zeros, D.device, "zeros", "weights")) != NP_OK) return st;
    struct Holder {
        np_w4* w = new np_w4();
        ~Holder() { delete w; }
    } hold;
    np_w4* const w = hold.w;
    w->desc = D;
    W4View& v = w->view;
    v.n_out = D.n_out;
    v.n_in = D.n_in;
    v.out_tiles = (D.n_out + kW4Outs - 1) / kW4Outs;
    v.chunks = (D.n_in + kW4Ins - 1) / kW4Ins;
    v.per_chunk = D.group < kW4Ins ? kW4Ins / D.group : 1;
    v.scale_words = D.scale_dtype == NP_F32 ? 2 : 1;
    const size_t all = (size_t)v.out_tiles * v.chunks, code_bytes = all * kW4TileBytes;
    const size_t scale_bytes = (all * v.per_chunk * kW4Outs * v.scale_words + 1) * sizeof(uint32_t);  // read two at a time
    if (hipMalloc((void**)&w->tiles, code_bytes) != hipSuccess || hipMalloc((void**)&w->scales, scale_bytes) != hipSuccess) {
        (void)hipGetLastError();
        return fail(NP_ENOMEM, "cannot allocate %zu bytes of weights", code_bytes + scale_bytes);
    }
    v.tiles = w->tiles;
    v.scales = w->scales;
    W4PackArgs a;
    a.codes = static_cast<const uint8_t*>(D.codes);
    a.scales = D.scales;
    a.zeros = D.zeros;
    a.tiles = w->tiles;
    a.scales_out = w->scales;
    a.n_out = D.n_out;
    a.n_in = D.n_in;
    a.out_tiles = v.out_tiles;
    a.chunks = v.chunks;
    a.per_chunk = v.per_chunk;
    a.group = D.group;
    a.groups = (D.n_in + D.group - 1) / D.group;
    a.scale_dtype = D.scale_dtype;
    NP_HIP(w4_prepare());
    NP_HIP(hipDeviceSynchronize());  // whatever stream filled the sources
    NP_HIP(launch_w4_pack(a, nullptr));
    NP_HIP(hipDeviceSynchronize());
    w->desc.codes = w->desc.scales = nullptr;  // read, not kept
    w->desc.zeros = nullptr;
    *out = w;
    hold.w = nullptr;
    return NP_OK;
}

np_status matvec(const np_w4* w, int64_t rows, const void* x, int32_t x_dtype, int64_t x_row, void* y, int32_t y_dtype, int64_t y_row, int32_t accumulate,
                 hipStream_t s) {
    if (!w) return fail(NP_EINVAL, "w must not be NULL");
    if (!known(x_dtype) || !known(y_dtype)) return fail(NP_EINVAL, "unknown dtype %d or %d", x_dtype, y_dtype);
    const np_w4_desc& D = w->desc;
    if (rows < 0 || rows > 1 << 20) return fail(NP_EINVAL, "rows=%lld must be in [0, 2^20]", (long long)rows);
    if (x_row == 0) x_row = D.n_in;
    if (y_row == 0) y_row = D.n_out;
    const int xb = elem_bytes(x_dtype), yb = elem_bytes(y_dtype);
    const bool some = rows > 0;  // without rows a tensor may have no address
    if ((some && !x) || !aligned16(x) || x_row < D.n_in || x_row > (int64_t)1 << 36 || x_row * xb % 16)
        return fail(NP_EINVAL, "x must be a 16-byte aligned device pointer, its stride %lld a multiple of 16 bytes of at least n_in=%d", (long long)x_row, D.n_in);
    if ((some && !y) || (uintptr_t)y % yb || y_row < D.n_out || y_row > (int64_t)1 << 36)
        return fail(NP_EINVAL, "y must be a device pointer aligned to its type, its stride %lld at least n_out=%d", (long long)y_row, D.n_out);
    if (accumulate != 0 && accumulate != 1) return fail(NP_EINVAL, "accumulate=%d must be 0 or 1", accumulate);
    const uint8_t* const x0 = static_cast<const uint8_t*>(x);
    const uint8_t* const y0 = static_cast<const uint8_t*>(y);
    if (some && x0 < y0 + ((rows - 1) * y_row + D.n_out) * yb && y0 < x0 + ((rows - 1) * x_row + D.n_in) * xb) {
        // Columns of the same rows may belong to both.
        const int64_t step = x_row * xb, off = step ? ((y0 - x0) % step + step) % step : 0;
        if (step != y_row * yb || off < (int64_t)D.n_in * xb || off + (int64_t)D.n_out * yb > step) return fail(NP_EINVAL, "x and y must not overlap");
    }
    // A launch has at most 2^32 - 1 threads along x: workgroups of 512 for 64 rows x 128 outputs each, at the most.
    if ((rows + 63) / 64 * ((D.n_out + 1023) / 1024 * 8) >= 1 << 23) return fail(NP_EINVAL, "%lld rows of %d outputs in one call are too many", (long long)rows, D.n_out);
    np_status st;
    if (x && (st = check_io_ptr(x, D.device, "x", "weights")) != NP_OK) return st;
    if (y && (st = check_io_ptr(y, D.device, "y", "weights")) != NP_OK) return st;
    if (!some) return NP_OK;
    W4Args a;
    a.w = w->view;
    a.x = x;
    a.y = y;
    a.rows = rows;
    a.x_row = x_row;
    a.y_row = y_row;
    a.y_dtype = y_dtype;
    a.accumulate = accumulate;
    DeviceGuard g(D.device);
    if (!g.ok) return fail(NP_EHIP, "hipSetDevice(%d) failed", D.device);
    NP_HIP(launch_w4(a, x_dtype, s));
    return NP_OK;
}

}  // namespace

extern "C" {

np_status np_w4_create(const np_w4_desc* desc, np_w4** out) {
    return guarded([&] { return create(desc, out); });
}

np_status np_w4_destroy(np_w4* w) {
    if (!w) return fail(NP_EINVAL, "w must not be NULL");
    DeviceGuard g(w->desc.device);
    CaptureGuard c;
    delete w;  // its first hipFree waits for the device
    return NP_OK;
}

np_status np_w4_matvec(const np_w4* w, int64_t rows, const void* x, int32_t x_dtype, int64_t x_row, void* y, int32_t y_dtype, int64_t y_row,
                       int32_t accumulate, void* stream) {
    return guarded([&] { return matvec(w, rows, x, x_dtype, x_row, y, y_dtype, y_row, accumulate, (hipStream_t)stream); });
}

}  // extern "C"
