// wkv_host.cuh -- host-side helpers that the C ABI's translation units share:
// error recording, argument checks and launches.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "../../include/wkv.h"

namespace wkv {
namespace host {

inline thread_local char g_last_cuda_error[256] = "";

constexpr int64_t kMaxElems = int64_t(1) << 62;
constexpr int kMaxDevices = 64;

// A workspace's first bytes: the error word that wkv_workspace_status() reads
// is among them, so what a call keeps of its own lies behind them.
constexpr size_t kHeader = 256;

inline int record_cuda(cudaError_t e) {
    if (e == cudaSuccess) return WKV_OK;
    std::snprintf(g_last_cuda_error, sizeof(g_last_cuda_error), "%s: %s", cudaGetErrorName(e),
                  cudaGetErrorString(e));
    return WKV_ERR_CUDA;
}

inline int check_launch() { return record_cuda(cudaPeekAtLastError()); }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// [p, p+bytes) intersects [q, q+qbytes)?
inline bool overlaps(const void* p, size_t bytes, const void* q, size_t qbytes) {
    if (p == nullptr || q == nullptr || bytes == 0 || qbytes == 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + qbytes && b < a + bytes;
}

inline bool mul_ok(int64_t a, int64_t b, int64_t c, int64_t* out) {
    if (a < 0 || b < 0 || c < 0) return false;
    __int128 p = static_cast<__int128>(a) * b * c;
    if (p >= kMaxElems) return false;
    *out = static_cast<int64_t>(p);
    return true;
}

inline size_t elem_bytes(int dtype) { return dtype == WKV_BF16 ? 2 : 4; }

// Limit of every wait on another CTA's result, and on the reverse delta rule's
// batches of tensor-core products: 1 s, or WKV_WAIT_LIMIT_NS (read
// once per process; used by the tests to make waits run out on purpose).
// Waits for a CTA's own TMA copies have a fixed limit (kCopyWaitNs).
inline uint64_t wait_limit_ns() {
    static const uint64_t v = []() -> uint64_t {
        const char* e = std::getenv("WKV_WAIT_LIMIT_NS");
        if (e != nullptr && *e != '\0') {
            char* end = nullptr;
            const unsigned long long x = std::strtoull(e, &end, 10);
            if (end != e) return x;
        }
        return 1000000000ull;
    }();
    return v;
}

// An argument's bytes, for the checks of a call with many of them.
struct Span {
    const void* p;
    size_t bytes, align;
};
// Outputs must overlap neither the inputs nor one another.
template <int NI, int NO>
int check_spans(const Span (&ins)[NI], const Span (&outs)[NO]) {
    for (const Span& s : ins)
        if (s.p && !aligned(s.p, s.align)) return WKV_ERR_ALIGN;
    for (const Span& s : outs)
        if (s.p && !aligned(s.p, s.align)) return WKV_ERR_ALIGN;
    for (int i = 0; i < NO; ++i) {
        for (const Span& s : ins)
            if (overlaps(outs[i].p, outs[i].bytes, s.p, s.bytes)) return WKV_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return WKV_ERR_ALIAS;
    }
    return WKV_OK;
}

// A launch that may begin while the stream's previous kernel ends (every
// kernel here waits for it before it touches memory).
template <typename... P, typename... A>
int launch(void (*kern)(P...), int64_t blocks, int threads, int smem, cudaStream_t st, A... args) {
    if (blocks <= 0) return WKV_OK;
    if (blocks > 0x7fffffffLL) return WKV_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return record_cuda(cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...));
}

// Dynamic shared memory above 48 KB, once per kernel and device.
template <typename K>
int allow_smem(K kern, int smem, bool (&ready)[kMaxDevices]) {
    int dev = 0;
    int rc = record_cuda(cudaGetDevice(&dev));
    if (rc != WKV_OK) return rc;
    if (dev < 0 || dev >= kMaxDevices) return WKV_ERR_CUDA;
    if (!ready[dev]) {
        rc = record_cuda(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
        if (rc != WKV_OK) return rc;
        ready[dev] = true;
    }
    return WKV_OK;
}

}  // namespace host
}  // namespace wkv
