// The HIP runtime and the kernels' launches as the host side of the key/value cache (np_kv.hip) sees them, without a
// device: compiled together with it by tests/test_kv_host_faults.py, so that failures can be forced and launches looked at.
#include <hip/hip_runtime_api.h>

#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <new>
#include <string>
#include <vector>

#include "kv_internal.hpp"
#include "np.h"
#include "np_host.hpp"

namespace {
std::string g_err;
int g_device = 0;            // current device
long g_news_left = -1;       // allocations until one fails (-1: none fails)
int g_set_fails = 0;         // hipSetDevice fails
int g_launches_left = -1;    // launches until one fails (-1: none fails)
long g_launches = 0;         // launches that were accepted
long g_wrong_device = 0;     // launches while another device was current
std::vector<int32_t> g_table;
}  // namespace

void* operator new(size_t n) {
    if (g_news_left == 0) throw std::bad_alloc();
    if (g_news_left > 0) --g_news_left;
    if (void* p = std::malloc(n ? n : 1)) return p;
    throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }

extern "C" {
void stub_fail_new(long after) { g_news_left = after; }
void stub_fail_set_device(int on) { g_set_fails = on; }
void stub_fail_launch(int after) { g_launches_left = after; }
long stub_launches() { return g_launches; }
long stub_wrong_device() { return g_wrong_device; }
int stub_device() { return g_device; }
const int32_t* stub_table() { return g_table.data(); }
const char* np_last_error() { return g_err.c_str(); }

hipError_t hipGetDeviceCount(int* n) { return *n = 2, hipSuccess; }
hipError_t hipGetDevice(int* d) { return *d = g_device, hipSuccess; }
hipError_t hipSetDevice(int d) {
    if (g_set_fails) return hipErrorInvalidDevice;
    return g_device = d, hipSuccess;
}
hipError_t hipMalloc(void** p, size_t n) { return *p = std::malloc(n), *p ? hipSuccess : hipErrorOutOfMemory; }
hipError_t hipFree(void* p) { return std::free(p), hipSuccess; }
hipError_t hipMemset(void* p, int v, size_t n) { return __builtin_memset(p, v, n), hipSuccess; }
hipError_t hipMemcpy(void* d, const void* s, size_t n, hipMemcpyKind) { return __builtin_memcpy(d, s, n), hipSuccess; }
hipError_t hipDeviceSynchronize() { return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "forced"; }
}

namespace np {

np_status fail(np_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    const long left = g_news_left;  // the text may allocate
    g_news_left = -1;
    g_err = buf;
    g_news_left = left;
    return st;
}
np_status check_io_ptr(const void*, int, const char*, const char*) { return NP_OK; }

// A launch: a grid dimension may have at most 2^32 - 1 threads.
static hipError_t launch(uint64_t threads_x) {
    if (g_device != 1) ++g_wrong_device;
    if (threads_x >> 32) return hipErrorInvalidConfiguration;
    if (g_launches_left == 0) return hipErrorLaunchFailure;
    if (g_launches_left > 0) --g_launches_left;
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_kv_append(const AppendArgs& a, int, hipStream_t) {
    return launch((uint64_t)a.b.item0[a.b.n] * a.kv.n_kv * 256);
}
hipError_t launch_kv_table(const TableArgs& a, hipStream_t) {
    const hipError_t e = launch(kTableEntries);
    if (e != hipSuccess) return e;
    for (int k = 0; k < a.n; ++k) {
        if ((size_t)a.at[k] >= g_table.size()) g_table.resize(a.at[k] + 1, -7);
        g_table[a.at[k]] = a.page[k];
    }
    return e;
}
hipError_t launch_kv_copy(const CopyArgs&, hipStream_t) { return launch(256); }
int attn_tile_rows(int dtype, int slabs) { return dtype != kF32 || slabs == 1 ? (slabs <= 3 ? 256 : 128) : 0; }
hipError_t launch_attn(const AttnArgs& a, int, hipStream_t) {
    return launch(a.part ? (uint64_t)a.b.item0[a.b.n] * 64 * kAttnWaves : (uint64_t)a.b.item0[a.b.n] * a.kv.n_kv * 512);
}
hipError_t attn_prepare() { return hipSuccess; }

}  // namespace np
