// wkv_delta.cu -- host side of the gated delta rule's entry points
// (wkv_delta_forward, wkv_delta_step, wkv_delta_backward): argument checks,
// the workspace's layout and the launches.
#include "wkv_delta_tc.cuh"
#include "wkv_host.cuh"

namespace {

using namespace wkv::host;
namespace d = wkv::delta;

// Walks in parts (Task in wkv_delta_mma.cuh) need walks that are not few and
// tokens for parts of kPartMin or more; kPartMax of them bound the work that
// the last wave leaves undone to an eighth of a walk.  4 x 8192 tokens of 80 heads
// of 64 (320 walks, 296 places): 1303 us whole, 1015 in 8 parts, 1035 in 32.
constexpr int64_t kPartMin = 256, kPartMax = 8, kSlotsMin = 148;

struct Parts {
    size_t ticket, done, hand, bytes;   // offsets, behind the header; 0 bytes: never in parts
};
// walks: heads times slices of their columns
Parts parts_layout(int64_t walks, int64_t states, int64_t T) {
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    Parts p{};
    if (walks <= kSlotsMin || T < 2 * kPartMin) return p;
    p.ticket = kHeader;
    p.done = p.ticket + 256;
    p.hand = p.done + up(size_t(walks) * 4);
    p.bytes = p.hand + up(size_t(states) * 4);
    return p;
}
int slices(int64_t N) { return N == 128 ? 2 : 1; }

using Walk = void (*)(d::Args);
// CTAs of `kern` that the GPU holds
int walk_slots(Walk kern, int threads, int smem, int64_t* slots) {
    int dev = 0, sms = 0, per = 0;
    int rc = record_cuda(cudaGetDevice(&dev));
    if (rc == WKV_OK) rc = record_cuda(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    if (rc == WKV_OK) rc = record_cuda(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, threads, size_t(smem)));
    *slots = int64_t(sms) * per;
    return rc;
}
// Do walks go in parts?  Where the share of the last wave's places that stay
// empty, of all waves', is above a tenth (a part costs a pipeline's fill).  Not in
// one wave that does not fill the GPU: 256 walks of 4096 tokens take 479 us in
// parts, 429 whole.
bool in_parts(int64_t walks, int64_t slots) {
    const int64_t waves = slots > 0 ? (walks + slots - 1) / slots : 0;
    return waves > 1 && (waves * slots - walks) * 10 > waves * slots;
}
int launch_parts(Walk kern, int64_t slots, int threads, int smem, d::Args a, char* ws, const Parts& p, cudaStream_t st) {
    const int64_t n = a.T / kPartMin < kPartMax ? a.T / kPartMin : kPartMax;
    a.part_len = ((a.T + n - 1) / n + d::kSegment - 1) / d::kSegment * d::kSegment;
    a.parts = (a.T + a.part_len - 1) / a.part_len;
    a.control = reinterpret_cast<d::Control*>(ws), a.wait_ns = wait_limit_ns();
    a.ticket = reinterpret_cast<uint32_t*>(ws + p.ticket);
    a.done = reinterpret_cast<uint32_t*>(ws + p.done);
    a.hand = reinterpret_cast<float*>(ws + p.hand);
    // the tickets and the parts that are done; the header stays
    const int rc = record_cuda(cudaMemsetAsync(ws + p.ticket, 0, p.hand - p.ticket, st));
    if (rc != WKV_OK) return rc;
    kern<<<dim3(unsigned(slots)), threads, smem, st>>>(a);
    return check_launch();
}

template <typename IO, int N, bool WANT_Y>
int launch_forward_parts(int64_t slots, const d::Args& a, char* ws, const Parts& p, cudaStream_t st) {
    using G = d::ForwardShape<IO, N, WANT_Y>;
    static bool ready[kMaxDevices] = {false};
    const auto kern = d::delta_forward_mma_kernel<IO, N, WANT_Y, true>;
    const int rc = allow_smem(kern, G::SMEM, ready);
    return rc != WKV_OK ? rc : launch_parts(kern, slots, G::THREADS, G::SMEM, a, ws, p, st);
}
// ws: parts_layout's bytes, or NULL
template <typename IO, int N>
int launch_forward(d::Args a, char* ws, const Parts& p, cudaStream_t st) {
    using G = d::ForwardShape<IO, N, true>;
    static bool ready[kMaxDevices] = {false};
    const auto kern = d::delta_forward_mma_kernel<IO, N, true, false>;
    const int64_t walks = a.B * a.H * G::SLICES;
    int64_t slots = 0;
    int rc = allow_smem(kern, G::SMEM, ready);
    if (rc == WKV_OK && ws != nullptr && p.bytes > 0) rc = walk_slots(kern, G::THREADS, G::SMEM, &slots);
    if (rc != WKV_OK) return rc;
    if (in_parts(walks, slots)) return launch_forward_parts<IO, N, true>(slots, a, ws, p, st);
    return launch(kern, walks, G::THREADS, G::SMEM, st, a);
}

// both walks of the reverse mode
template <typename IO, int N>
int launch_walks(d::Args a, char* ws, const Parts& p, cudaStream_t st) {
    using F = d::ForwardShape<IO, N, false>;
    using R = d::ReverseShape<IO, N>;
    static_assert(F::THREADS == R::THREADS && F::SMEM <= R::SMEM && F::SLICES == R::SLICES, "one kernel for both");
    static bool ready[2][kMaxDevices] = {{false}};
    const auto kern = d::delta_walks_kernel<IO, N>;
    const auto reverse = d::delta_reverse_mma_kernel<IO, N>;
    const int64_t walks = a.B * a.H * R::SLICES;
    int64_t slots = 0;
    int rc = allow_smem(kern, R::SMEM, ready[0]);
    if (rc == WKV_OK) rc = allow_smem(reverse, R::SMEM, ready[1]);
    if (rc == WKV_OK && p.bytes > 0) rc = walk_slots(reverse, R::THREADS, R::SMEM, &slots);
    if (rc != WKV_OK) return rc;
    if (!in_parts(walks, slots)) return launch(kern, 2 * walks, R::THREADS, R::SMEM, st, a);
    rc = launch_forward_parts<IO, N, false>(slots, a, ws, p, st);
    return rc != WKV_OK ? rc : launch_parts(reverse, slots, R::THREADS, R::SMEM, a, ws, p, st);
}

template <typename IO, int N>
int launch_segments(const d::Args& a, cudaStream_t st) {
    static bool ready[kMaxDevices] = {false};
    const int64_t segments = a.B * a.H * ((a.T + d::kSegment - 1) / d::kSegment);
    if constexpr (d::kTcSegments<IO, N>) {
        using G = d::TcSegment;
        const int rc = allow_smem(d::delta_segment_tc_kernel, G::SMEM, ready);
        return rc != WKV_OK ? rc : launch(d::delta_segment_tc_kernel, segments, G::THREADS, G::SMEM, st, a);
    } else {
        using G = d::SegmentShape<IO, N>;
        const auto kern = d::delta_segment_kernel<IO, N>;
        const int rc = allow_smem(kern, G::SMEM, ready);
        return rc != WKV_OK ? rc : launch(kern, segments, G::THREADS, G::SMEM, st, a);
    }
}

struct Layout {
    size_t e, du, s_seg, d_seg, drh, dkh, bytes;
};

// share: several value heads to a key head
Layout layout(int64_t B, int64_t T, int64_t H, int64_t N, bool share) {
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t val = up(size_t(B) * T * H * N * 4), heads = size_t(B) * H;
    const size_t borders = heads * (size_t((T + d::kSegment - 1) / d::kSegment) + 1);
    Layout l{};
    const size_t parts = parts_layout(B * H * slices(N), B * H * N * N, T).bytes;
    l.e = parts > 0 ? parts : kHeader;
    l.du = l.e + val;
    l.s_seg = l.du + val;
    l.d_seg = l.s_seg + up(borders * N * N * 4);
    l.drh = l.d_seg + up(borders * N * N * 4);
    l.dkh = l.drh + (share ? val : 0);
    l.bytes = l.dkh + (share ? val : 0);
    return l;
}

template <typename IO, int N>
int run_backward(const d::Args& a, char* ws, const Parts& p, cudaStream_t st) {
    int rc = launch_walks<IO, N>(a, ws, p, st);
    if (rc == WKV_OK) rc = launch_segments<IO, N>(a, st);
    if (rc == WKV_OK && a.H != a.Hk)
        rc = launch(d::delta_share_kernel<IO, N>, (a.B * a.T * a.Hk * (N / 4) + 255) / 256, 256, 0, st, a);
    return rc;
}

template <typename IO, int N>
int run_step(int64_t heads, int64_t Hk, int64_t H, const float* w, const float* beta, const void* r, const void* k,
             const void* v, float* state, void* y, cudaStream_t st) {
    constexpr int CL = N == 128 ? 4 : 8, NW = 4, PARTS = N / (CL * 4);
    return launch(d::delta_step_kernel<IO, N, CL, NW>, (heads * PARTS + NW - 1) / NW, NW * 32, 0, st, heads, Hk, H, w,
                  beta, static_cast<const IO*>(r), static_cast<const IO*>(k), static_cast<const IO*>(v), state,
                  static_cast<IO*>(y), aligned(state, 16));
}

// sizes: the counts of keys, values, per-head scalars and states, or an error
struct Sizes {
    int64_t keys, values, scalars, states;
};
int sizes(int64_t lead0, int64_t lead1, int64_t nstates, int64_t Hk, int64_t H, int64_t N, Sizes* s) {
    if (lead0 < 0 || lead1 < 0 || nstates < 0 || (N != 32 && N != 64 && N != 128) || Hk <= 0 || H <= 0 || H % Hk != 0)
        return WKV_ERR_SHAPE;
    int64_t tokens = 0, hn = 0;
    if (!mul_ok(lead0, lead1, 1, &tokens) || !mul_ok(H, N, 1, &hn)) return WKV_ERR_SHAPE;
    if (!mul_ok(tokens, hn, 8, &s->values) || !mul_ok(nstates, hn, N * 8, &s->states)) return WKV_ERR_SHAPE;
    s->values /= 8;
    s->states /= 8;
    s->keys = tokens * Hk * N;
    s->scalars = tokens * H;
    return WKV_OK;
}

// f(type tag, head size) for the call's type and head size
template <typename F>
int with_type(int dtype, int64_t N, F f) {
    auto pick = [&](auto tag) {
        if (N == 32) return f(tag, std::integral_constant<int, 32>{});
        if (N == 64) return f(tag, std::integral_constant<int, 64>{});
        return f(tag, std::integral_constant<int, 128>{});
    };
    return dtype == WKV_F32 ? pick(float{}) : pick(__nv_bfloat16{});
}

// the state passed through when there is no token
int pass_state(const float* in, float* out, size_t bytes, cudaStream_t st) {
    if (out == nullptr || out == in || bytes == 0) return WKV_OK;
    if (!aligned(out, 4) || !aligned(in, 4)) return WKV_ERR_ALIGN;
    if (overlaps(in, bytes, out, bytes)) return WKV_ERR_ALIAS;
    if (in) return record_cuda(cudaMemcpyAsync(out, in, bytes, cudaMemcpyDeviceToDevice, st));
    return record_cuda(cudaMemsetAsync(out, 0, bytes, st));
}

}  // namespace

extern "C" {

int wkv_delta_forward(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, int dtype, const float* w,
                      const float* beta, const void* r, const void* k, const void* v, const float* state_in, void* y,
                      float* state_out, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (dtype != WKV_F32 && dtype != WKV_BF16) return WKV_ERR_DTYPE;
    Sizes n{};
    int rc = sizes(B, T, B, Hk, H, N, &n);
    if (rc != WKV_OK) return rc;
    if (B == 0) return WKV_OK;
    const size_t eb = elem_bytes(dtype), sb = size_t(n.states) * 4;
    if (T == 0) return pass_state(state_in, state_out, sb, stream);
    if (!w || !beta || !r || !k || !v || !y) return WKV_ERR_NULLPTR;
    const Span ins[] = {{w, size_t(n.scalars) * 4, 4}, {beta, size_t(n.scalars) * 4, 4}, {r, size_t(n.keys) * eb, eb},
                        {k, size_t(n.keys) * eb, eb}, {v, size_t(n.values) * eb, eb},
                        {state_in == state_out ? nullptr : state_in, sb, 4}};
    // a workspace that is too small is not touched
    const Parts p = parts_layout(B * H * slices(N), n.states, T);
    if (p.bytes == 0 || workspace_bytes < p.bytes) workspace = nullptr;
    const Span outs[] = {{y, size_t(n.values) * eb, eb}, {state_out, sb, 4}, {workspace, p.bytes, 256}};
    rc = check_spans(ins, outs);
    if (rc != WKV_OK) return rc;
    if (workspace && overlaps(workspace, p.bytes, state_in, sb)) return WKV_ERR_ALIAS;
    d::Args a{};
    a.B = B, a.T = T, a.Hk = Hk, a.H = H;
    a.w = w, a.beta = beta, a.r = r, a.k = k, a.v = v, a.s_in = state_in, a.y = y, a.s_out = state_out;
    a.vec = aligned(r, 16) && aligned(k, 16) && aligned(v, 16) && aligned(y, 16);
    rc = with_type(dtype, N, [&](auto tag, auto size) {
        return launch_forward<decltype(tag), decltype(size)::value>(a, static_cast<char*>(workspace), p, stream);
    });
    return rc != WKV_OK ? rc : check_launch();
}

size_t wkv_delta_forward_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t N) {
    Sizes n{};
    if (sizes(B, T, B, 1, H, N, &n) != WKV_OK) return 0;
    return parts_layout(B * H * slices(N), n.states, T).bytes;
}

int wkv_delta_step(int64_t L, int64_t B, int64_t Hk, int64_t H, int64_t N, int dtype, const float* w,
                   const float* beta, const void* r, const void* k, const void* v, float* state, void* y,
                   cudaStream_t stream) {
    if (dtype != WKV_F32 && dtype != WKV_BF16) return WKV_ERR_DTYPE;
    Sizes n{};
    int rc = sizes(L, B, L >= 0 && B >= 0 && L < (int64_t(1) << 31) && B < (int64_t(1) << 31) ? L * B : -1, Hk, H, N, &n);
    if (rc != WKV_OK) return rc;
    if (L == 0 || B == 0) return WKV_OK;
    if (!w || !beta || !r || !k || !v || !state || !y) return WKV_ERR_NULLPTR;
    const size_t eb = elem_bytes(dtype);
    const Span ins[] = {{w, size_t(n.scalars) * 4, 4}, {beta, size_t(n.scalars) * 4, 4}, {r, size_t(n.keys) * eb, eb},
                        {k, size_t(n.keys) * eb, eb}, {v, size_t(n.values) * eb, eb}};
    const Span outs[] = {{y, size_t(n.values) * eb, eb}, {state, size_t(n.states) * 4, 4}};
    rc = check_spans(ins, outs);
    if (rc != WKV_OK) return rc;
    rc = with_type(dtype, N, [&](auto tag, auto size) {
        return run_step<decltype(tag), decltype(size)::value>(L * B * H, Hk, H, w, beta, r, k, v, state, y, stream);
    });
    return rc != WKV_OK ? rc : check_launch();
}

size_t wkv_delta_backward_workspace_bytes(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N) {
    Sizes n{};
    if (sizes(B, T, B, Hk, H, N, &n) != WKV_OK || B == 0 || T == 0) return 0;
    return layout(B, T, H, N, H != Hk).bytes;
}

int wkv_delta_backward(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, int dtype, const float* w,
                       const float* beta, const void* r, const void* k, const void* v, const float* state_in,
                       const void* dy, const float* dstate_out, void* dr, void* dk, void* dv, float* dw, float* dbeta,
                       float* dstate_in, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (dtype != WKV_F32 && dtype != WKV_BF16) return WKV_ERR_DTYPE;
    Sizes n{};
    int rc = sizes(B, T, B, Hk, H, N, &n);
    if (rc != WKV_OK) return rc;
    if (B == 0) return WKV_OK;
    const size_t eb = elem_bytes(dtype), sb = size_t(n.states) * 4;
    if (T == 0) {
        if (dstate_in == dstate_out && dstate_in != nullptr) return WKV_ERR_ALIAS;
        return pass_state(dstate_out, dstate_in, sb, stream);
    }
    if (!w || !beta || !r || !k || !v || !dy || !dr || !dk || !dv || !dw || !dbeta) return WKV_ERR_NULLPTR;
    const Layout l = layout(B, T, H, N, H != Hk);
    if (workspace == nullptr || workspace_bytes < l.bytes) return WKV_ERR_WORKSPACE;
    const size_t kb = size_t(n.keys) * eb, vb = size_t(n.values) * eb, pb = size_t(n.scalars) * 4;
    const Span ins[] = {{w, pb, 4}, {beta, pb, 4}, {r, kb, eb}, {k, kb, eb}, {v, vb, eb}, {state_in, sb, 4},
                        {dy, vb, eb}, {dstate_out, sb, 4}};
    const Span outs[] = {{dr, kb, eb}, {dk, kb, eb}, {dv, vb, eb}, {dw, pb, 4}, {dbeta, pb, 4}, {dstate_in, sb, 4},
                         {workspace, l.bytes, 256}};
    rc = check_spans(ins, outs);
    if (rc != WKV_OK) return rc;
    char* ws = static_cast<char*>(workspace);
    auto f = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
    d::Args a{};
    a.B = B, a.T = T, a.Hk = Hk, a.H = H;
    a.w = w, a.beta = beta, a.r = r, a.k = k, a.v = v, a.dy = dy, a.s_in = state_in, a.ds_out = dstate_out;
    a.dv = dv, a.ds_in = dstate_in;
    a.dr = dr, a.dk = dk, a.dw = dw, a.dbeta = dbeta;
    a.e = f(l.e), a.du = f(l.du), a.s_seg = f(l.s_seg), a.d_seg = f(l.d_seg);
    a.drh = f(l.drh), a.dkh = f(l.dkh);
    a.control = reinterpret_cast<d::Control*>(ws), a.wait_ns = wait_limit_ns();
    a.vec = aligned(r, 16) && aligned(k, 16) && aligned(v, 16) && aligned(dy, 16) && aligned(dv, 16) &&
            aligned(dr, 16) && aligned(dk, 16);
    rc = with_type(dtype, N, [&](auto tag, auto size) {
        return run_backward<decltype(tag), decltype(size)::value>(a, ws, parts_layout(B * H * slices(N), n.states, T), stream);
    });
    return rc != WKV_OK ? rc : check_launch();
}

int wkv_delta_status(int clear, cudaStream_t stream) {
    uint32_t lost = 0;
    int rc = record_cuda(cudaMemcpyFromSymbolAsync(&lost, d::g_lost, sizeof(lost), 0, cudaMemcpyDeviceToHost, stream));
    if (rc == WKV_OK) rc = record_cuda(cudaStreamSynchronize(stream));
    if (rc == WKV_OK && clear && lost) {
        static const uint32_t none = 0;
        rc = record_cuda(cudaMemcpyToSymbolAsync(d::g_lost, &none, sizeof(none), 0, cudaMemcpyHostToDevice, stream));
    }
    return rc != WKV_OK ? rc : lost ? WKV_ERR_TIMEOUT : WKV_OK;
}

}  // extern "C"
