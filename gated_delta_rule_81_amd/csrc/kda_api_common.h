// kda_api_common.h -- host-side argument checks, device checks and the debug
// mode shared by the sources that implement the C ABI (kda_api.cpp,
// layer_api.cpp).  Everything is local to the including source.
#pragma once

#include "kda.h"

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <atomic>
#include <vector>

namespace {

constexpr int kMaxDevices = 64;
std::atomic<int> g_device_ok[kMaxDevices];  // 0 unknown, 1 gfx950, -1 other

bool aligned16(const void *p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void *p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

struct Range {
    const void *p;
    uint64_t bytes;
};

bool overlap(const Range &a, const Range &b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Compute units of the current device (cached per device; 0 if unknown).
std::atomic<int> g_device_cus[kMaxDevices];
int device_cus() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    int n = g_device_cus[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
            return 0;
        g_device_cus[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

int check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return KDA_ERR_DEVICE;
    if (dev >= kMaxDevices) return KDA_ERR_DEVICE;
    int st = g_device_ok[dev].load(std::memory_order_relaxed);
    if (st == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return KDA_ERR_DEVICE;
        st = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
        g_device_ok[dev].store(st, std::memory_order_relaxed);
    }
    return st == 1 ? KDA_OK : KDA_ERR_DEVICE;
}

// Debug mode (environment variable KDA_DEBUG set to a value other than "0",
// read at every call): packed-sequence offsets are copied to the host and
// checked before the launch, and every call waits for its stream and reports
// any failure of its kernels as KDA_ERR_LAUNCH, with a line on stderr naming
// the entry point.  Off by default: calls stay asynchronous.
bool debug_mode() {
    const char *e = getenv("KDA_DEBUG");
    return e && e[0] && strcmp(e, "0") != 0;
}

// Debug mode: cu_seqlens must hold num_seqs + 1 offsets starting at 0,
// non-decreasing and ending at total.  Returns KDA_OK or KDA_ERR_SHAPE.
int debug_check_offsets(const int32_t *cu_seqlens, int64_t num_seqs, int64_t total,
                        hipStream_t stream, const char *where) {
    if (!cu_seqlens) return KDA_OK;
    std::vector<int32_t> cu((size_t)num_seqs + 1);
    if (hipStreamSynchronize(stream) != hipSuccess ||
        hipMemcpy(cu.data(), cu_seqlens, cu.size() * 4, hipMemcpyDeviceToHost) != hipSuccess) {
        fprintf(stderr, "[kda debug] %s: cannot read cu_seqlens\n", where);
        return KDA_ERR_LAUNCH;
    }
    bool ok = cu[0] == 0 && cu[(size_t)num_seqs] == total;
    for (size_t i = 0; ok && i < (size_t)num_seqs; ++i) ok = cu[i] <= cu[i + 1];
    if (!ok) {
        fprintf(stderr, "[kda debug] %s: cu_seqlens is not 0 = c0 <= c1 <= ... <= cN = %lld\n",
                where, (long long)total);
        return KDA_ERR_SHAPE;
    }
    return KDA_OK;
}

// The status of a call whose launches returned `rc` (0 = queued): in debug
// mode also wait for the stream and check what its kernels did.
int launch_status(int rc, hipStream_t stream, const char *where) {
    if (rc != 0) {
        if (debug_mode()) fprintf(stderr, "[kda debug] %s: launch failed\n", where);
        return KDA_ERR_LAUNCH;
    }
    if (debug_mode()) {
        const hipError_t e = hipStreamSynchronize(stream);
        const hipError_t l = hipGetLastError();
        if (e != hipSuccess || l != hipSuccess) {
            fprintf(stderr, "[kda debug] %s: %s\n", where,
                    hipGetErrorString(e != hipSuccess ? e : l));
            return KDA_ERR_LAUNCH;
        }
    }
    return KDA_OK;
}

}  // namespace
