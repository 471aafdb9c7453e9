// wkv_norm.cu -- host side of the group norm's entry points (wkv_group_norm,
// wkv_group_norm_backward): argument checks, the choice of a lane's vector
// and the launches.
#include "wkv_host.cuh"
#include "wkv_norm.cuh"

#include <cmath>

namespace {

using namespace wkv::host;
namespace nm = wkv::norm;

constexpr int kMaxE = 16;           // channels of a lane in registers; larger groups take large_kernel
constexpr int64_t kLargePer = 64;   // tokens a thread of large_params_kernel sums

struct Plan {
    int per, v;        // channels of a vector, vectors of a lane; v == 0: large_kernel
    int lpg, lpg_log2;
    int64_t slots, chunks;
    int span;
    size_t bytes;      // reverse mode's workspace
};

// elem: bytes of a value; align: largest power of two, up to 16, that divides
// every tensor's address
Plan plan(int64_t rows, int64_t C, int64_t group, int elem, int align, bool bwd) {
    Plan p{};
    p.per = 16 / elem;
    while (p.per > 1 && (group % p.per != 0 || p.per * elem > align)) p.per /= 2;
    const int64_t vecs = group / p.per;
    const int64_t groups = C / group;
    const int maxv = kMaxE / p.per < 8 ? kMaxE / p.per : 8;
    if (vecs > 32 * maxv) {
        p.per = 1;
        p.chunks = (rows + kLargePer - 1) / kLargePer;
        p.bytes = bwd ? size_t(rows) * groups * 8 + size_t(p.chunks) * C * 8 + 512 : 0;
        return p;
    }
    p.lpg = 1;
    while (p.lpg < 32 && p.lpg < vecs) p.lpg *= 2, ++p.lpg_log2;
    p.v = 1;
    while (p.v * p.lpg < vecs) p.v *= 2;
    p.slots = (groups * p.lpg + 31) / 32 * 32;
    // as many CTAs as the machine holds a few times over (forward), or twice
    // (reverse: a chunk's partial sums cost 8 bytes a channel), and no more
    const int64_t fill = int64_t(148) * 256 * (bwd ? 4 : 24);
    int64_t span = (rows * p.slots + fill - 1) / fill;
    const int64_t most = bwd ? 256 : 32;
    span = span < 1 ? 1 : span > most ? most : span;
    p.span = int(span);
    p.chunks = (rows + p.span - 1) / p.span;
    p.bytes = bwd ? size_t(p.chunks) * C * 8 : 0;
    return p;
}

template <typename R>
int launch_ring(void (*kern)(nm::Args), int64_t blocks, const nm::Args& a, cudaStream_t st) {
    int rc = WKV_OK;
    if constexpr (R::SMEM > 48 * 1024)   // groups of over 8 channels a lane only: set at each call
        rc = record_cuda(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, R::SMEM));
    return rc != WKV_OK ? rc : launch(kern, blocks, 256, R::SMEM, st, a);
}

template <typename IO, int PER, int V, bool GATE>
int launch_backward(const nm::Args& a, int64_t blocks, cudaStream_t st) {
    using R = nm::Ring<IO, PER, V, GATE, true>;
    if (a.act == nm::kSilu) return launch_ring<R>(nm::backward_kernel<IO, PER, V, GATE, nm::kSilu>, blocks, a, st);
    if (a.act == nm::kSigmoid) return launch_ring<R>(nm::backward_kernel<IO, PER, V, GATE, nm::kSigmoid>, blocks, a, st);
    return launch_ring<R>(nm::backward_kernel<IO, PER, V, GATE, nm::kNone>, blocks, a, st);
}

template <typename IO, int PER, int V, bool BWD>
int launch_small(const nm::Args& a, int64_t chunks, cudaStream_t st) {
    const int64_t blocks = (chunks * a.slots + 255) / 256;
    if constexpr (BWD)
        return a.gate ? launch_backward<IO, PER, V, true>(a, blocks, st) : launch_backward<IO, PER, V, false>(a, blocks, st);
    else
        return a.gate ? launch_ring<nm::Ring<IO, PER, V, true, false>>(nm::forward_kernel<IO, PER, V, true>, blocks, a, st)
                      : launch_ring<nm::Ring<IO, PER, V, false, false>>(nm::forward_kernel<IO, PER, V, false>, blocks, a, st);
}

template <typename IO, int PER, bool BWD>
int launch_v(const nm::Args& a, const Plan& p, cudaStream_t st) {
    switch (p.v) {
        case 1: return launch_small<IO, PER, 1, BWD>(a, p.chunks, st);
        case 2: return launch_small<IO, PER, 2, BWD>(a, p.chunks, st);
        case 4:
            if constexpr (PER * 4 <= kMaxE) return launch_small<IO, PER, 4, BWD>(a, p.chunks, st);
            break;
        case 8:
            if constexpr (PER * 8 <= kMaxE) return launch_small<IO, PER, 8, BWD>(a, p.chunks, st);
            break;
    }
    return WKV_ERR_SHAPE;
}

template <typename IO, bool BWD>
int launch_per(const nm::Args& a, const Plan& p, cudaStream_t st) {
    switch (p.per) {
        case 1: return launch_v<IO, 1, BWD>(a, p, st);
        case 2: return launch_v<IO, 2, BWD>(a, p, st);
        case 4: return launch_v<IO, 4, BWD>(a, p, st);
        default:
            if constexpr (sizeof(IO) == 2) return launch_v<IO, 8, BWD>(a, p, st);
            return WKV_ERR_SHAPE;
    }
}

template <typename IO, bool BWD>
int run(nm::Args& a, const Plan& p, int64_t groups, float* ws, float* dweight, float* dbias, cudaStream_t st) {
    const bool params = dweight != nullptr || dbias != nullptr;
    float* part = ws;
    int rc;
    if (p.v > 0) {
        a.part = params ? part : nullptr;
        rc = launch_per<IO, BWD>(a, p, st);
    } else {
        if (params) {
            a.part = ws;   // the groups' statistics, then the partial sums
            part = ws + (size_t(a.rows) * groups * 2 + 63) / 64 * 64;
        }
        const int64_t n = a.rows * groups, most = 148 * 8 * 4;
        rc = launch(nm::large_kernel<IO, BWD>, n < most ? n : most, 256, 0, st, a, groups);
        if (rc == WKV_OK && params) {
            for (int64_t c0 = 0; rc == WKV_OK && c0 < p.chunks; c0 += 32768) {
                const int64_t nc = p.chunks - c0 < 32768 ? p.chunks - c0 : 32768;
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3(unsigned((a.C + 127) / 128), unsigned(nc));
                cfg.blockDim = dim3(128);
                cfg.stream = st;
                nm::Args s = a;
                const int64_t r0 = c0 * kLargePer;
                s.rows = a.rows - r0;
                s.x = static_cast<const IO*>(a.x) + r0 * a.C;
                s.dy = static_cast<const IO*>(a.dy) + r0 * a.C;
                s.gate = a.gate ? static_cast<const IO*>(a.gate) + r0 * a.C : nullptr;
                rc = record_cuda(cudaLaunchKernelEx(&cfg, nm::large_params_kernel<IO>, s, groups,
                                                    static_cast<const float*>(ws + r0 * groups * 2),
                                                    part + c0 * 2 * a.C, kLargePer));
            }
        }
    }
    if (rc == WKV_OK && params)
        rc = launch(nm::params_kernel, (a.C + 31) / 32, 1024, 0, st, a.C, p.chunks, part, dweight, dbias);
    return rc;
}

int shape_ok(int64_t rows, int64_t C, int64_t G, int act, float eps) {
    int64_t n = 0;
    if (!mul_ok(rows, C, 8, &n) || G <= 0 || C % G != 0 || C / (G > 0 ? G : 1) > (1 << 30)) return WKV_ERR_SHAPE;
    if (act < 0 || act > 2 || !(eps > 0.f) || !std::isfinite(eps)) return WKV_ERR_SHAPE;
    return WKV_OK;
}

int common_align(const void* const* p, int n) {
    int a = 16;
    for (int i = 0; i < n; ++i)
        while (p[i] && !aligned(p[i], size_t(a))) a /= 2;
    return a;
}

}  // namespace

extern "C" {

int wkv_group_norm(int64_t rows, int64_t C, int64_t G, int dtype, int act, float eps, const void* x,
                   const float* weight, const float* bias, const void* gate, void* y, cudaStream_t stream) {
    if (dtype != WKV_F32 && dtype != WKV_BF16) return WKV_ERR_DTYPE;
    int rc = shape_ok(rows, C, G, act, eps);
    if (rc != WKV_OK) return rc;
    if (rows == 0 || C == 0) return WKV_OK;
    if (!x || !y) return WKV_ERR_NULLPTR;
    const size_t eb = elem_bytes(dtype), n = size_t(rows) * C * eb, pb = size_t(C) * 4;
    const Span ins[] = {{x, n, eb}, {weight, pb, 4}, {bias, pb, 4}, {gate, n, eb}};
    const Span outs[] = {{y, n, eb}};
    rc = check_spans(ins, outs);
    if (rc != WKV_OK) return rc;
    const void* ptrs[] = {x, gate, y};
    const Plan p = plan(rows, C, C / G, int(eb), common_align(ptrs, 3), false);
    nm::Args a{};
    a.rows = rows, a.C = C, a.group = int(C / G), a.lpg = p.lpg, a.lpg_log2 = p.lpg_log2, a.slots = p.slots;
    a.span = p.span, a.act = act, a.eps = eps, a.inv_group = 1.f / float(C / G);
    a.x = x, a.gate = gate, a.weight = weight, a.bias = bias, a.y = y;
    rc = dtype == WKV_F32 ? run<float, false>(a, p, G, nullptr, nullptr, nullptr, stream)
                          : run<__nv_bfloat16, false>(a, p, G, nullptr, nullptr, nullptr, stream);
    return rc != WKV_OK ? rc : check_launch();
}

size_t wkv_group_norm_backward_workspace_bytes(int64_t rows, int64_t C, int64_t G, int dtype) {
    if (dtype != WKV_F32 && dtype != WKV_BF16) return 0;
    if (shape_ok(rows, C, G, 0, 1.f) != WKV_OK || rows == 0 || C == 0) return 0;
    // any alignment the call's tensors may have
    size_t most = 0;
    for (int align = 16; align >= int(elem_bytes(dtype)); align /= 2) {
        const size_t b = plan(rows, C, C / G, int(elem_bytes(dtype)), align, true).bytes;
        if (b > most) most = b;
    }
    return most > 0 ? kHeader + most : 0;
}

int wkv_group_norm_backward(int64_t rows, int64_t C, int64_t G, int dtype, int act, float eps, const void* x,
                            const float* weight, const float* bias, const void* gate, const void* dy, void* dx,
                            float* dweight, float* dbias, void* dgate, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
    if (dtype != WKV_F32 && dtype != WKV_BF16) return WKV_ERR_DTYPE;
    int rc = shape_ok(rows, C, G, act, eps);
    if (rc != WKV_OK) return rc;
    if (C == 0) return WKV_OK;
    const size_t eb = elem_bytes(dtype), n = size_t(rows) * C * eb, pb = size_t(C) * 4;
    if (rows > 0 && (!x || !dy || !dx || (gate && !dgate))) return WKV_ERR_NULLPTR;
    if (!gate && dgate) return WKV_ERR_NULLPTR;
    const bool params = dweight != nullptr || dbias != nullptr;
    const size_t need = params ? wkv_group_norm_backward_workspace_bytes(rows, C, G, dtype) : 0;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return WKV_ERR_WORKSPACE;
    const Span ins[] = {{x, n, eb}, {weight, pb, 4}, {bias, pb, 4}, {gate, n, eb}, {dy, n, eb}};
    const Span outs[] = {{dx, n, eb}, {dweight, pb, 4}, {dbias, pb, 4}, {dgate, n, eb},
                         {need ? workspace : nullptr, need, 256}};
    rc = check_spans(ins, outs);
    if (rc != WKV_OK) return rc;
    if (rows == 0) {
        if (dweight) rc = record_cuda(cudaMemsetAsync(dweight, 0, pb, stream));
        if (rc == WKV_OK && dbias) rc = record_cuda(cudaMemsetAsync(dbias, 0, pb, stream));
        return rc;
    }
    const void* ptrs[] = {x, gate, dy, dx, dgate};
    const Plan p = plan(rows, C, C / G, int(eb), common_align(ptrs, 5), true);
    nm::Args a{};
    a.rows = rows, a.C = C, a.group = int(C / G), a.lpg = p.lpg, a.lpg_log2 = p.lpg_log2, a.slots = p.slots;
    a.span = p.span, a.act = act, a.eps = eps, a.inv_group = 1.f / float(C / G);
    a.x = x, a.gate = gate, a.weight = weight, a.bias = bias, a.dy = dy, a.dx = dx, a.dgate = dgate;
    float* ws = need > 0 ? static_cast<float*>(workspace) + kHeader / 4 : nullptr;
    rc = dtype == WKV_F32 ? run<float, true>(a, p, G, ws, dweight, dbias, stream)
                          : run<__nv_bfloat16, true>(a, p, G, ws, dweight, dbias, stream);
    return rc != WKV_OK ? rc : check_launch();
}

}  // extern "C"
