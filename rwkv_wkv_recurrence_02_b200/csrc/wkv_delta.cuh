// wkv_delta.cuh -- the gated delta rule: forward walk and the four walks of
// its reverse mode.
//
// Per head, with states S (N x N, key channel i, value channel j), decay
// a_t = e^{-w_t} and learning rate beta_t:
//   e_t = v_t - a_t S_{t-1}^T k_t          the error of the decayed state's read at k_t
//   S_t = a_t S_{t-1} + k_t (beta_t e_t)^T
//   y_t = S_t^T r_t
// Reverse mode, D_t the gradient of S_t (y_t's own part included):
//   D_t = Dn_t + r_t dy_t^T,  du_t = D_t^T k_t,  dv_t = beta_t du_t,
//   Dn_{t-1} = a_t (D_t - k_t dv_t^T),
//   dr_t = S_t dy_t,  dk_t = D_t (beta_t e_t) - a_t S_{t-1} dv_t,
//   dbeta_t = du_t . e_t,  dw_t = -<Dn_{t-1}, S_{t-1}>,
//   <Dn_{t-1}, S_{t-1}> = <Dn_t, S_t> + r_t . dr_t - dv_t . v_t.
//
// Every walk is a recurrence over tokens on a matrix X whose columns (forward
// and D walks) or rows (the walks that form dr and dk) are independent, so
// a warp takes a slice of them with the whole reduction axis and no two
// warps exchange anything.  A walk is float32 multiply-adds on the CUDA
// cores: the state has to stay at float32 accuracy, for which the tensor
// cores would need each operand in three bfloat16 pieces.  What bounds a walk
// is the fp32 pipe.
//
// Decay without a multiply per state value: within a block of TB tokens the
// state is kept as X / g_t, g_t the product of the block's decays up to t, and
// the factors go into the staged vectors.  g is a product of at most TB
// rounded factors, as exact as multiplying the state each token would be.  A
// block whose product falls below kMinScale (strong decays, a reset) multiplies
// the state at every token instead.
#pragma once

#include <type_traits>

#include "wkv_common.cuh"

namespace wkv {
namespace delta {

// smallest product of decays a block carries outside its state: the scaled
// state stays below 2^80 times its size, far from float32's range
constexpr float kMinScale = 8.271806125530277e-25f;   // 2^-80
// tokens between the states the reverse mode keeps for dw
constexpr int kCheck = 64;

template <typename IO>
__device__ __forceinline__ float to_f32(IO x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// ---------------------------------------------------------------------------
// Staging: TB rows of W elements (row t at base + t * stride), read into
// registers one block ahead and written to shared memory as float32 times a
// factor for each row.  vec: 16-byte loads (base and stride allow them).
// ---------------------------------------------------------------------------
template <typename IO, int TB, int W, int THREADS>
struct Stage {
    static constexpr int PER = 16 / int(sizeof(IO));
    static constexpr int ROWV = W / PER;
    static constexpr int VECS = TB * ROWV;
    static constexpr int PT = (VECS + THREADS - 1) / THREADS;
    uint4 raw[PT];

    __device__ __forceinline__ void load(const IO* base, int64_t stride, int nt, bool vec, int tid) {
#pragma unroll
        for (int n = 0; n < PT; ++n) {
            const int i = tid + n * THREADS;
            const int t = i / ROWV, c = (i % ROWV) * PER;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (i < VECS && t < nt) {
                const IO* p = base + t * stride + c;
                if (vec) {
                    x = __ldg(reinterpret_cast<const uint4*>(p));
                } else {
                    uint32_t e[4];
                    if constexpr (sizeof(IO) == 4) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) e[j] = __float_as_uint(__ldg(reinterpret_cast<const float*>(p) + j));
                    } else {
                        const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
                        for (int j = 0; j < 4; ++j) e[j] = uint32_t(__ldg(q + 2 * j)) | uint32_t(__ldg(q + 2 * j + 1)) << 16;
                    }
                    x = make_uint4(e[0], e[1], e[2], e[3]);
                }
            }
            raw[n] = x;
        }
    }
    // row t times the factor held by lane t of the warp (all lanes call)
    __device__ __forceinline__ void store(float* dst, float fac, int tid) const {
#pragma unroll
        for (int n = 0; n < PT; ++n) {
            const int i = tid + n * THREADS;
            const int t = i / ROWV, c = (i % ROWV) * PER;
            const float f = __shfl_sync(0xffffffffu, fac, t < TB ? t : 0);
            if (VECS % THREADS == 0 || i < VECS) {
                const uint32_t e[4] = {raw[n].x, raw[n].y, raw[n].z, raw[n].w};
                float4* o = reinterpret_cast<float4*>(dst + t * W + c);
                if constexpr (sizeof(IO) == 4) {
                    o[0] = make_float4(__uint_as_float(e[0]) * f, __uint_as_float(e[1]) * f, __uint_as_float(e[2]) * f,
                                       __uint_as_float(e[3]) * f);
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        o[j] = make_float4(__uint_as_float(e[2 * j] << 16) * f, __uint_as_float(e[2 * j] & 0xffff0000u) * f,
                                           __uint_as_float(e[2 * j + 1] << 16) * f,
                                           __uint_as_float(e[2 * j + 1] & 0xffff0000u) * f);
                }
            }
        }
    }
};

// ---------------------------------------------------------------------------
// A warp's slice of a state: CW = (32 / RG) * CC independent lines, the
// reduction axis (N) over RG lanes.  Lane (g, cl) holds, of lines
// cl * CC + c, the positions j * 4 RG + 4 g + e: a 16-byte shared load of all
// RG lanes is one contiguous run, so the lanes' banks differ.  Packed pairs
// along the reduction axis.
// ---------------------------------------------------------------------------
template <int N, int RG, int CC>
struct Tile {
    static constexpr int CG = 32 / RG;
    static constexpr int R = N / RG;
    static constexpr int J = R / 4;
    static constexpr int CW = CG * CC;
    static_assert(R % 4 == 0 && CC % 2 == 0, "tile shape");
    F2 s[CC][R / 2];

    struct Vec4 { F2 lo, hi; };
    static __device__ __forceinline__ Vec4 at(const float* x, int j, int g) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(x + j * 4 * RG + 4 * g);
        return Vec4{F2{v.x}, F2{v.y}};
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int c = 0; c < CC; ++c)
#pragma unroll
            for (int i = 0; i < R / 2; ++i) s[c][i] = f2s(0.f);
    }
    // X(line, pos) at S[pos * N + line] (TRANS false) or S[line * N + pos]
    template <bool TRANS>
    __device__ __forceinline__ void load(const float* S, int line0, int g) {
#pragma unroll
        for (int c = 0; c < CC; ++c)
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
                const int pos = (i / 2) * 4 * RG + 4 * g + (i % 2) * 2;
                s[c][i] = TRANS ? f2(S[(line0 + c) * N + pos], S[(line0 + c) * N + pos + 1])
                                : f2(S[pos * N + line0 + c], S[(pos + 1) * N + line0 + c]);
            }
    }
    template <bool TRANS>
    __device__ __forceinline__ void store(float* S, int line0, int g) const {
#pragma unroll
        for (int c = 0; c < CC; ++c)
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
                const int pos = (i / 2) * 4 * RG + 4 * g + (i % 2) * 2;
                const float a = f2lo(s[c][i]), b = f2hi(s[c][i]);
                S[TRANS ? (line0 + c) * N + pos : pos * N + line0 + c] = a;
                S[TRANS ? (line0 + c) * N + pos + 1 : (pos + 1) * N + line0 + c] = b;
            }
    }
    // the slice as it lies in registers (coalesced; for the reverse mode's own use)
    __device__ __forceinline__ void store_raw(float* p, int lane) const {
#pragma unroll
        for (int c = 0; c < CC; ++c)
#pragma unroll
            for (int i = 0; i < R / 2; ++i)
                reinterpret_cast<unsigned long long*>(p)[(c * (R / 2) + i) * 32 + lane] = s[c][i].v;
    }
    __device__ __forceinline__ float dot_raw(const float* p, int lane) const {
        F2 acc = f2s(0.f);
#pragma unroll
        for (int c = 0; c < CC; ++c)
#pragma unroll
            for (int i = 0; i < R / 2; ++i)
                acc = fma2(s[c][i], F2{__ldcg(reinterpret_cast<const unsigned long long*>(p) + (c * (R / 2) + i) * 32 + lane)},
                           acc);
        return f2lo(acc) + f2hi(acc);
    }
    __device__ __forceinline__ void scale(float f) {
        const F2 ff = f2s(f);
#pragma unroll
        for (int c = 0; c < CC; ++c)
#pragma unroll
            for (int i = 0; i < R / 2; ++i) s[c][i] = mul2(s[c][i], ff);
    }
    // this lane's part of X x for each line
    __device__ __forceinline__ void dot(const float* x, int g, float (&o)[CC]) const {
        F2 acc[CC];
#pragma unroll
        for (int c = 0; c < CC; ++c) acc[c] = f2s(0.f);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const Vec4 v = at(x, j, g);
#pragma unroll
            for (int c = 0; c < CC; ++c) {
                acc[c] = fma2(s[c][2 * j], v.lo, acc[c]);
                acc[c] = fma2(s[c][2 * j + 1], v.hi, acc[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < CC; ++c) o[c] = f2lo(acc[c]) + f2hi(acc[c]);
    }
    __device__ __forceinline__ void add(const float* x, int g, const float (&f)[CC]) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const Vec4 v = at(x, j, g);
#pragma unroll
            for (int c = 0; c < CC; ++c) {
                const F2 ff = f2s(f[c]);
                s[c][2 * j] = fma2(v.lo, ff, s[c][2 * j]);
                s[c][2 * j + 1] = fma2(v.hi, ff, s[c][2 * j + 1]);
            }
        }
    }
    // sums over the RG lanes of a line, all lanes
    static __device__ __forceinline__ void all_sum(float (&x)[CC]) {
#pragma unroll
        for (int o = 1; o < RG; o *= 2)
#pragma unroll
            for (int c = 0; c < CC; ++c) x[c] += __shfl_xor_sync(0xffffffffu, x[c], o);
    }
    // sums over the RG lanes of a line, each lane left with OUT of them:
    // lines out_line() .. + OUT - 1 in x[0 .. OUT)
    static constexpr int OUT = CC > RG ? CC / RG : 1;
    static __device__ __forceinline__ void spread_sum(float (&x)[CC], int g) {
        int n = CC;
#pragma unroll
        for (int o = 1; o < RG; o *= 2) {
            if (n > 1) {
                n /= 2;
#pragma unroll
                for (int c = 0; c < CC / 2; ++c)
                    if (c < n) {
                        const float keep = (g & o) ? x[n + c] : x[c], send = (g & o) ? x[c] : x[n + c];
                        x[c] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                    }
            } else {
                x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
            }
        }
    }
    static __device__ __forceinline__ int out_line(int g) {
        int n = CC, l = 0;
#pragma unroll
        for (int o = 1; o < RG; o *= 2)
            if (n > 1) {
                n /= 2;
                if (g & o) l += n;
            }
        return l;
    }
    // whether this lane's sums are the ones to store (the others hold copies)
    static __device__ __forceinline__ bool out_lane(int g) { return CC >= RG || g < CC; }
};

// ---------------------------------------------------------------------------
// Decays of a block, one token to a lane (lanes of TB and above repeat lane
// TB - 1's).
// ---------------------------------------------------------------------------
struct Decay {
    float a, scale, total;   // a_t; product of the decays carried to t; the whole block's
    bool slow;
};
// REV: scale_t = product of the decays after t; else of those up to t.
template <int TB, bool REV>
__device__ __forceinline__ Decay block_decay(float w, int lane) {
    Decay d;
    d.a = expf(-w);
    float x = d.a;
#pragma unroll
    for (int o = 1; o < TB; o *= 2) {
        const float y = REV ? __shfl_down_sync(0xffffffffu, x, o) : __shfl_up_sync(0xffffffffu, x, o);
        if (REV ? lane + o < TB : lane >= o) x *= y;
    }
    d.total = __shfl_sync(0xffffffffu, x, REV ? 0 : TB - 1);
    if (REV) {
        const float after = __shfl_down_sync(0xffffffffu, x, 1);
        x = lane < TB - 1 ? after : 1.f;
    }
    // NaN decays take the slow way too, and reach the state there
    d.slow = !(d.total >= kMinScale);
    d.scale = d.slow ? 1.f : x;
    return d;
}

struct Args {
    int64_t B, T, Hk, H;
    const float* w;      // (B, T, H)
    const float* beta;   // (B, T, H)
    const void* r;       // (B, T, Hk, N)
    const void* k;
    const void* v;       // (B, T, H, N)
    const void* dy;
    const float* s_in;   // (B, H, N, N)
    void* y;
    float* s_out;
    const float* ds_out;
    void* dv;
    float* ds_in;
    // reverse mode's workspace
    float* e;            // (B, T, H, N)
    float* du;
    float* dr;           // (B, T, H, N), per value head
    float* dk;           // the state's part
    float* dk2;          // the gradient state's part
    float* check;        // (B, H, n + 1, N, N), n = ceil(T / kCheck)
    float* phi;          // (B, H, n + 1, slots)
    bool vec;            // 16-byte loads of every tensor in the I/O type
};

// ---------------------------------------------------------------------------
// Forward walk, value columns.  WANT_Y: outputs; otherwise the errors e for
// the reverse mode.  Three multiply-adds for each state value and token
// (two without y).  The outputs of token t - 1 are formed between the two
// halves of token t's read, so that their multiply-adds cover the shuffles.
// ---------------------------------------------------------------------------
template <typename IO, int N, int RG, int CC, int NW, int TB, bool WANT_Y>
struct ForwardShape {
    using T = Tile<N, RG, CC>;
    static constexpr int MC = NW * T::CW, SLICES = N / MC, THREADS = NW * 32;
    static constexpr int STEP = TB * (N * (WANT_Y ? 2 : 1) + MC + 4);   // floats of one stage
    static constexpr int SMEM = 2 * STEP * 4;
};

template <typename IO, int N, int RG, int CC, int NW, int TB, bool WANT_Y>
__global__ void __launch_bounds__(NW * 32) delta_forward_kernel(const Args a) {
    using G = ForwardShape<IO, N, RG, CC, NW, TB, WANT_Y>;
    using Tl = typename G::T;
    extern __shared__ __align__(16) float smem[];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int g = lane % RG, cl = lane / RG;
    const int64_t head = blockIdx.x / G::SLICES;
    const int slice = int(blockIdx.x % G::SLICES) * G::MC;
    const int64_t b = head / a.H, h = head % a.H, hk = h / (a.H / a.Hk);
    const int line0 = warp * Tl::CW + cl * CC;   // within the slice
    const int64_t ks = a.Hk * N, vs = a.H * N;
    const IO* kp = static_cast<const IO*>(a.k) + (b * a.T * a.Hk + hk) * N;
    const IO* rp = static_cast<const IO*>(a.r) + (b * a.T * a.Hk + hk) * N;
    const IO* vp = static_cast<const IO*>(a.v) + (b * a.T * a.H + h) * N + slice;
    const float* wp = a.w + b * a.T * a.H + h;
    const float* bp = a.beta + b * a.T * a.H + h;
    pdl_begin();

    Tl X;
    if (a.s_in != nullptr)
        X.template load<false>(a.s_in + head * N * N, slice + line0, g);
    else
        X.zero();

    Stage<IO, TB, N, G::THREADS> sk, sr;
    Stage<IO, TB, G::MC, G::THREADS> sv;
    float w = 0.f, beta = 0.f;
    auto fetch = [&](int64_t t0) {
        const int nt = a.T - t0 < TB ? int(a.T - t0) : TB;
        sk.load(kp + t0 * ks, ks, nt, a.vec, tid);
        if constexpr (WANT_Y) sr.load(rp + t0 * ks, ks, nt, a.vec, tid);
        sv.load(vp + t0 * vs, vs, nt, a.vec, tid);
        w = lane < nt ? __ldg(wp + (t0 + lane) * a.H) : 0.f;
        beta = lane < nt ? __ldg(bp + (t0 + lane) * a.H) : 0.f;
    };
    auto stage = [&](float* buf) {
        const Decay d = block_decay<TB, false>(w, lane);
        sk.store(buf, 1.f, tid);
        if constexpr (WANT_Y) sr.store(buf + TB * N, d.scale, tid);
        sv.store(buf + TB * N * (WANT_Y ? 2 : 1), 1.f, tid);
        if (warp == 0 && lane < TB)
            reinterpret_cast<float4*>(buf + TB * (N * (WANT_Y ? 2 : 1) + G::MC))[lane] =
                make_float4(d.scale, beta / d.scale, d.a, 0.f);
        return d;
    };
    auto give = [&](int64_t t, const float (&x)[CC]) {   // y of token t, after spread_sum
        if (Tl::out_lane(g)) {
            IO* yp = static_cast<IO*>(a.y) + (b * a.T + t) * vs + h * N + slice + line0 + Tl::out_line(g);
#pragma unroll
            for (int c = 0; c < Tl::OUT; ++c) put(yp + c, x[c]);
        }
    };

    fetch(0);
    Decay d = stage(smem);
    __syncthreads();
    int cur = 0;
    for (int64_t t0 = 0; t0 < a.T; t0 += TB) {
        const int nt = a.T - t0 < TB ? int(a.T - t0) : TB;
        const bool more = t0 + TB < a.T;
        if (more) fetch(t0 + TB);
        const float* bk = smem + cur * G::STEP;
        const float* br = bk + TB * N;
        const float* bv = bk + TB * N * (WANT_Y ? 2 : 1);
        const float4* bs = reinterpret_cast<const float4*>(bv + TB * G::MC);
        float q[CC];
        auto token = [&](int t, auto slow, auto first) {
            const float4 sc = bs[t];
            if constexpr (decltype(slow)::value) {
                if constexpr (WANT_Y && !decltype(first)::value) X.dot(br + (t - 1) * N, g, q);
                X.scale(sc.z);
            }
            float p[CC], u[CC];
            X.dot(bk + t * N, g, p);
            if constexpr (!decltype(slow)::value && WANT_Y && !decltype(first)::value) X.dot(br + (t - 1) * N, g, q);
            Tl::all_sum(p);
#pragma unroll
            for (int c = 0; c < CC; ++c) {
                const float e = fmaf(-(decltype(slow)::value ? 1.f : sc.x), p[c], bv[t * G::MC + line0 + c]);
                u[c] = sc.y * e;
                if constexpr (!WANT_Y) {
                    if (g == c % RG) a.e[(b * a.T + t0 + t) * vs + h * N + slice + line0 + c] = e;
                }
            }
            X.add(bk + t * N, g, u);
            if constexpr (WANT_Y && !decltype(first)::value) {
                Tl::spread_sum(q, g);
                give(t0 + t - 1, q);
            }
        };
        using Yes = std::true_type;
        using No = std::false_type;
        if (!d.slow) {
            token(0, No{}, Yes{});
#pragma unroll 1
            for (int t = 1; t < nt; ++t) token(t, No{}, No{});
        } else {
            token(0, Yes{}, Yes{});
#pragma unroll 1
            for (int t = 1; t < nt; ++t) token(t, Yes{}, No{});
        }
        if constexpr (WANT_Y) {
            X.dot(br + (nt - 1) * N, g, q);
            Tl::spread_sum(q, g);
            give(t0 + nt - 1, q);
        }
        if (!d.slow) X.scale(d.total);
        cur ^= 1;
        if (more) d = stage(smem + cur * G::STEP);
        __syncthreads();
    }
    if (WANT_Y && a.s_out != nullptr) X.template store<false>(a.s_out + head * N * N, slice + line0, g);
}

// ---------------------------------------------------------------------------
// Reverse walk of the gradient state, value columns: du, dv and the initial
// state's gradient.  The outer product of the next token's r and dy goes in
// while the shuffles of this token's read are under way (both are sums).
// ---------------------------------------------------------------------------
template <typename IO, int N, int RG, int CC, int NW, int TB>
struct ReverseShape {
    using T = Tile<N, RG, CC>;
    static constexpr int MC = NW * T::CW, SLICES = N / MC, THREADS = NW * 32;
    static constexpr int STEP = TB * (2 * N + MC + 4);
    static constexpr int SMEM = 2 * STEP * 4;
};

template <typename IO, int N, int RG, int CC, int NW, int TB>
__global__ void __launch_bounds__(NW * 32) delta_reverse_kernel(const Args a) {
    using G = ReverseShape<IO, N, RG, CC, NW, TB>;
    using Tl = typename G::T;
    extern __shared__ __align__(16) float smem[];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int g = lane % RG, cl = lane / RG;
    const int64_t head = blockIdx.x / G::SLICES;
    const int slice = int(blockIdx.x % G::SLICES) * G::MC;
    const int64_t b = head / a.H, h = head % a.H, hk = h / (a.H / a.Hk);
    const int line0 = warp * Tl::CW + cl * CC;
    const int64_t ks = a.Hk * N, vs = a.H * N;
    const IO* kp = static_cast<const IO*>(a.k) + (b * a.T * a.Hk + hk) * N;
    const IO* rp = static_cast<const IO*>(a.r) + (b * a.T * a.Hk + hk) * N;
    const IO* yp = static_cast<const IO*>(a.dy) + (b * a.T * a.H + h) * N + slice;
    const float* wp = a.w + b * a.T * a.H + h;
    const float* bp = a.beta + b * a.T * a.H + h;
    pdl_begin();

    Tl X;
    if (a.ds_out != nullptr)
        X.template load<false>(a.ds_out + head * N * N, slice + line0, g);
    else
        X.zero();

    Stage<IO, TB, N, G::THREADS> sk, sr;
    Stage<IO, TB, G::MC, G::THREADS> sy;
    float w = 0.f, beta = 0.f;
    auto fetch = [&](int64_t t0) {
        const int nt = a.T - t0 < TB ? int(a.T - t0) : TB;
        sk.load(kp + t0 * ks, ks, nt, a.vec, tid);
        sr.load(rp + t0 * ks, ks, nt, a.vec, tid);
        sy.load(yp + t0 * vs, vs, nt, a.vec, tid);
        w = lane < nt ? __ldg(wp + (t0 + lane) * a.H) : 0.f;
        beta = lane < nt ? __ldg(bp + (t0 + lane) * a.H) : 0.f;
    };
    auto stage = [&](float* buf) {
        const Decay d = block_decay<TB, true>(w, lane);
        sk.store(buf, 1.f, tid);
        sr.store(buf + TB * N, 1.f, tid);
        sy.store(buf + 2 * TB * N, 1.f / d.scale, tid);
        if (warp == 0 && lane < TB)
            reinterpret_cast<float4*>(buf + TB * (2 * N + G::MC))[lane] = make_float4(d.scale, beta, d.a, 0.f);
        return d;
    };

    const int64_t last = (a.T - 1) / TB * TB;
    fetch(last);
    Decay d = stage(smem);
    __syncthreads();
    int cur = 0;
    for (int64_t t0 = last; t0 >= 0; t0 -= TB) {
        const int nt = a.T - t0 < TB ? int(a.T - t0) : TB;
        if (t0 > 0) fetch(t0 - TB);
        const float* bk = smem + cur * G::STEP;
        const float* br = bk + TB * N;
        const float* by = br + TB * N;
        const float4* bs = reinterpret_cast<const float4*>(by + TB * G::MC);
        auto enter = [&](int t) {   // the outer product r_t dy_t^T
            float f[CC];
#pragma unroll
            for (int c = 0; c < CC; ++c) f[c] = by[t * G::MC + line0 + c];
            X.add(br + t * N, g, f);
        };
        enter(nt - 1);
#pragma unroll 1
        for (int t = nt - 1; t >= 0; --t) {
            const float4 sc = bs[t];
            float p[CC], f[CC];
            X.dot(bk + t * N, g, p);
            if (!d.slow && t > 0) enter(t - 1);
            Tl::all_sum(p);
#pragma unroll
            for (int c = 0; c < CC; ++c) {
                f[c] = -sc.y * p[c];
                if (g == c % RG) {
                    const int64_t at = (b * a.T + t0 + t) * vs + h * N + slice + line0 + c;
                    const float du = (d.slow ? 1.f : sc.x) * p[c];
                    a.du[at] = du;
                    put(static_cast<IO*>(a.dv) + at, sc.y * du);
                }
            }
            X.add(bk + t * N, g, f);
            if (d.slow) {
                X.scale(sc.z);
                if (t > 0) enter(t - 1);
            }
        }
        if (!d.slow) X.scale(d.total);
        cur ^= 1;
        if (t0 > 0) d = stage(smem + cur * G::STEP);
        __syncthreads();
    }
    if (a.ds_in != nullptr) X.template store<false>(a.ds_in + head * N * N, slice + line0, g);
}

// ---------------------------------------------------------------------------
// Key rows: the state's walk again, now with e known, for dr and the state's
// part of dk; keeps the states between chunks of kCheck tokens for dw.
// ---------------------------------------------------------------------------
template <typename IO, int N, int RG, int CC, int NW, int TB>
struct RowShape {
    using T = Tile<N, RG, CC>;
    static constexpr int MC = NW * T::CW, SLICES = N / MC, THREADS = NW * 32;
    static constexpr int STEP = TB * (3 * N + 2 * MC + 4);
    static constexpr int SMEM = 2 * STEP * 4;
    static constexpr int SLOTS = N / T::CW;
};

template <typename IO, int N, int RG, int CC, int NW, int TB>
__global__ void __launch_bounds__(NW * 32) delta_state_rows_kernel(const Args a) {
    using G = RowShape<IO, N, RG, CC, NW, TB>;
    using Tl = typename G::T;
    static_assert(kCheck % TB == 0, "blocks meet the chunk borders");
    extern __shared__ __align__(16) float smem[];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int g = lane % RG, cl = lane / RG;
    const int64_t head = blockIdx.x / G::SLICES;
    const int slice = int(blockIdx.x % G::SLICES) * G::MC;
    const int64_t b = head / a.H, h = head % a.H, hk = h / (a.H / a.Hk);
    const int line0 = warp * Tl::CW + cl * CC;
    const int64_t ks = a.Hk * N, vs = a.H * N;
    const int64_t base = (b * a.T * a.H + h) * N;
    const IO* kp = static_cast<const IO*>(a.k) + (b * a.T * a.Hk + hk) * N + slice;
    const IO* yp = static_cast<const IO*>(a.dy) + base;
    const float* wp = a.w + b * a.T * a.H + h;
    const float* bp = a.beta + b * a.T * a.H + h;
    const int64_t nchunk = (a.T + kCheck - 1) / kCheck;
    float* ck = a.check + head * (nchunk + 1) * N * N + (slice / Tl::CW + warp) * (N * Tl::CW);
    pdl_begin();

    Tl X;
    if (a.s_in != nullptr)
        X.template load<true>(a.s_in + head * N * N, slice + line0, g);
    else
        X.zero();

    Stage<float, TB, N, G::THREADS> se, sd;
    Stage<IO, TB, N, G::THREADS> sy;
    Stage<IO, TB, G::MC, G::THREADS> sk;
    float w = 0.f, beta = 0.f;
    auto fetch = [&](int64_t t0) {
        const int nt = a.T - t0 < TB ? int(a.T - t0) : TB;
        se.load(a.e + base + t0 * vs, vs, nt, true, tid);
        sd.load(a.du + base + t0 * vs, vs, nt, true, tid);
        sy.load(yp + t0 * vs, vs, nt, a.vec, tid);
        sk.load(kp + t0 * ks, ks, nt, a.vec, tid);
        w = lane < nt ? __ldg(wp + (t0 + lane) * a.H) : 0.f;
        beta = lane < nt ? __ldg(bp + (t0 + lane) * a.H) : 0.f;
    };
    auto stage = [&](float* buf) {
        const Decay d = block_decay<TB, false>(w, lane);
        se.store(buf, beta / d.scale, tid);
        sd.store(buf + TB * N, beta * d.scale, tid);
        sy.store(buf + 2 * TB * N, d.scale, tid);
        sk.store(buf + 3 * TB * N, 1.f, tid);
        if (warp == 0 && lane < TB) buf[TB * (3 * N + 2 * G::MC) + lane] = d.a;
        return d;
    };

    fetch(0);
    Decay d = stage(smem);
    __syncthreads();
    int cur = 0;
    for (int64_t t0 = 0; t0 < a.T; t0 += TB) {
        const int nt = a.T - t0 < TB ? int(a.T - t0) : TB;
        const bool more = t0 + TB < a.T;
        if (more) fetch(t0 + TB);
        if (t0 % kCheck == 0) X.store_raw(ck + (t0 / kCheck) * N * N, lane);
        const float* bu = smem + cur * G::STEP;
        const float* bd = bu + TB * N;
        const float* by = bd + TB * N;
        const float* bk = by + TB * N;
        const float* ba = bk + TB * 2 * G::MC;
#pragma unroll 1
        for (int t = 0; t < nt; ++t) {
            if (d.slow) X.scale(ba[t]);
            float o1[CC], o2[CC], f[CC];
            X.dot(bd + t * N, g, o1);
#pragma unroll
            for (int c = 0; c < CC; ++c) f[c] = bk[t * G::MC + line0 + c];
            X.add(bu + t * N, g, f);
            X.dot(by + t * N, g, o2);
            Tl::spread_sum(o1, g);
            Tl::spread_sum(o2, g);
            if (Tl::out_lane(g)) {
                const int64_t at = base + (t0 + t) * vs + slice + line0 + Tl::out_line(g);
#pragma unroll
                for (int c = 0; c < Tl::OUT; ++c) {
                    a.dk[at + c] = -o1[c];
                    a.dr[at + c] = o2[c];
                }
            }
        }
        if (!d.slow) X.scale(d.total);
        cur ^= 1;
        if (more) d = stage(smem + cur * G::STEP);
        __syncthreads();
    }
    X.store_raw(ck + nchunk * N * N, lane);
}

// ---------------------------------------------------------------------------
// Key rows of the gradient state, reverse: the other part of dk, and at each
// chunk border the inner product <Dn, S> that dw continues from.
// ---------------------------------------------------------------------------
template <typename IO, int N, int RG, int CC, int NW, int TB>
__global__ void __launch_bounds__(NW * 32) delta_grad_rows_kernel(const Args a) {
    using G = RowShape<IO, N, RG, CC, NW, TB>;
    using Tl = typename G::T;
    extern __shared__ __align__(16) float smem[];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int g = lane % RG, cl = lane / RG;
    const int64_t head = blockIdx.x / G::SLICES;
    const int slice = int(blockIdx.x % G::SLICES) * G::MC;
    const int64_t b = head / a.H, h = head % a.H, hk = h / (a.H / a.Hk);
    const int line0 = warp * Tl::CW + cl * CC;
    const int64_t ks = a.Hk * N, vs = a.H * N;
    const int64_t base = (b * a.T * a.H + h) * N;
    const IO* kp = static_cast<const IO*>(a.k) + (b * a.T * a.Hk + hk) * N + slice;
    const IO* rp = static_cast<const IO*>(a.r) + (b * a.T * a.Hk + hk) * N + slice;
    const IO* yp = static_cast<const IO*>(a.dy) + base;
    const float* wp = a.w + b * a.T * a.H + h;
    const float* bp = a.beta + b * a.T * a.H + h;
    const int64_t nchunk = (a.T + kCheck - 1) / kCheck;
    const int slot = slice / Tl::CW + warp;
    const float* ck = a.check + head * (nchunk + 1) * N * N + slot * (N * Tl::CW);
    float* phi = a.phi + head * (nchunk + 1) * G::SLOTS + slot;
    pdl_begin();

    Tl X;
    auto border = [&](int64_t c) {
        float x = X.dot_raw(ck + c * N * N, lane);
#pragma unroll
        for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) phi[c * G::SLOTS] = x;
    };
    if (a.ds_out != nullptr) {
        X.template load<true>(a.ds_out + head * N * N, slice + line0, g);
        border(nchunk);
    } else {
        X.zero();
        if (lane == 0) phi[nchunk * G::SLOTS] = 0.f;
    }

    Stage<float, TB, N, G::THREADS> se, sd;
    Stage<IO, TB, N, G::THREADS> sy;
    Stage<IO, TB, G::MC, G::THREADS> sk, sr;
    float w = 0.f, beta = 0.f;
    auto fetch = [&](int64_t t0) {
        const int nt = a.T - t0 < TB ? int(a.T - t0) : TB;
        se.load(a.e + base + t0 * vs, vs, nt, true, tid);
        sd.load(a.du + base + t0 * vs, vs, nt, true, tid);
        sy.load(yp + t0 * vs, vs, nt, a.vec, tid);
        sk.load(kp + t0 * ks, ks, nt, a.vec, tid);
        sr.load(rp + t0 * ks, ks, nt, a.vec, tid);
        w = lane < nt ? __ldg(wp + (t0 + lane) * a.H) : 0.f;
        beta = lane < nt ? __ldg(bp + (t0 + lane) * a.H) : 0.f;
    };
    auto stage = [&](float* buf) {
        const Decay d = block_decay<TB, true>(w, lane);
        se.store(buf, beta * d.scale, tid);
        sd.store(buf + TB * N, -beta / d.scale, tid);
        sy.store(buf + 2 * TB * N, 1.f / d.scale, tid);
        sk.store(buf + 3 * TB * N, 1.f, tid);
        sr.store(buf + 3 * TB * N + TB * G::MC, 1.f, tid);
        if (warp == 0 && lane < TB) buf[TB * (3 * N + 2 * G::MC) + lane] = d.a;
        return d;
    };

    const int64_t last = (a.T - 1) / TB * TB;
    fetch(last);
    Decay d = stage(smem);
    __syncthreads();
    int cur = 0;
    for (int64_t t0 = last; t0 >= 0; t0 -= TB) {
        const int nt = a.T - t0 < TB ? int(a.T - t0) : TB;
        if (t0 > 0) fetch(t0 - TB);
        const float* bu = smem + cur * G::STEP;
        const float* bd = bu + TB * N;
        const float* by = bd + TB * N;
        const float* bk = by + TB * N;
        const float* br = bk + TB * G::MC;
        const float* ba = br + TB * G::MC;
#pragma unroll 1
        for (int t = nt - 1; t >= 0; --t) {
            float o[CC], f[CC];
#pragma unroll
            for (int c = 0; c < CC; ++c) f[c] = br[t * G::MC + line0 + c];
            X.add(by + t * N, g, f);
            X.dot(bu + t * N, g, o);
#pragma unroll
            for (int c = 0; c < CC; ++c) f[c] = bk[t * G::MC + line0 + c];
            X.add(bd + t * N, g, f);
            if (d.slow) X.scale(ba[t]);
            Tl::spread_sum(o, g);
            if (Tl::out_lane(g)) {
                const int64_t at = base + (t0 + t) * vs + slice + line0 + Tl::out_line(g);
#pragma unroll
                for (int c = 0; c < Tl::OUT; ++c) a.dk2[at + c] = o[c];
            }
        }
        if (!d.slow) X.scale(d.total);
        if (t0 % kCheck == 0) border(t0 / kCheck);
        cur ^= 1;
        if (t0 > 0) d = stage(smem + cur * G::STEP);
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Per token: dr and dk of a key head (the sums over the value heads that share
// it), dbeta, and the token's term of dw's sum.  One warp per (sequence,
// token, key head).
// ---------------------------------------------------------------------------
template <typename IO, int N>
__global__ void __launch_bounds__(256) delta_tokens_kernel(const Args a, IO* __restrict__ dr, IO* __restrict__ dk,
                                                           float* __restrict__ dbeta, float* __restrict__ term) {
    constexpr int E = N / 32;
    const int lane = threadIdx.x % 32;
    const int64_t id = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
    pdl_begin();
    if (id >= a.B * a.T * a.Hk) return;
    const int64_t bt = id / a.Hk, hk = id % a.Hk;
    const int share = int(a.H / a.Hk);
    float rr[E], sr[E], sk[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        rr[i] = to_f32(static_cast<const IO*>(a.r)[id * N + i * 32 + lane]);
        sr[i] = sk[i] = 0.f;
    }
    for (int s = 0; s < share; ++s) {
        const int64_t hh = bt * a.H + hk * share + s;
        float x1 = 0.f, x2 = 0.f, x3 = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int64_t at = hh * N + i * 32 + lane;
            const float gr = a.dr[at], du = a.du[at];
            sr[i] += gr;
            sk[i] += a.dk[at] + a.dk2[at];
            x1 = fmaf(rr[i], gr, x1);
            x2 = fmaf(du, to_f32(static_cast<const IO*>(a.v)[at]), x2);
            x3 = fmaf(du, a.e[at], x3);
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2) {
            x1 += __shfl_xor_sync(0xffffffffu, x1, o);
            x2 += __shfl_xor_sync(0xffffffffu, x2, o);
            x3 += __shfl_xor_sync(0xffffffffu, x3, o);
        }
        if (lane == 0) {
            dbeta[hh] = x3;
            term[hh] = x1 - a.beta[hh] * x2;
        }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
        put(dr + id * N + i * 32 + lane, sr[i]);
        put(dk + id * N + i * 32 + lane, sk[i]);
    }
}

// dw of a chunk: the sum <Dn, S> from the chunk's end backwards; its first
// token's is the border's own.  One thread per (sequence, chunk, head).
template <int SLOTS>
__global__ void __launch_bounds__(128) delta_dw_kernel(const Args a, const float* __restrict__ term, float* __restrict__ dw) {
    const int64_t nchunk = (a.T + kCheck - 1) / kCheck;
    const int64_t id = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    pdl_begin();
    if (id >= a.B * nchunk * a.H) return;
    const int64_t h = id % a.H, c = id / a.H % nchunk, b = id / a.H / nchunk;
    const float* phi = a.phi + ((b * a.H + h) * (nchunk + 1) + c) * SLOTS;
    float first = 0.f, x = 0.f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) first += phi[s], x += phi[SLOTS + s];
    const int64_t t0 = c * kCheck, t1 = t0 + kCheck < a.T ? t0 + kCheck : a.T;
    for (int64_t t = t1 - 1; t > t0; --t) {
        const int64_t at = (b * a.T + t) * a.H + h;
        x += term[at];
        // a state that nothing is left of has no gradient, whatever the sum's rounding left
        dw[at] = expf(-a.w[at]) == 0.f ? 0.f : -x;
    }
    dw[(b * a.T + t0) * a.H + h] = -first;
}

// ---------------------------------------------------------------------------
// One token for L layers (B sequences, H heads each): the state is read once,
// held in registers and written once, which is what bounds it.
// ---------------------------------------------------------------------------
template <typename IO, int N, int CL, int NW>
__global__ void __launch_bounds__(NW * 32)
delta_step_kernel(int64_t heads, int64_t Hk, int64_t H, const float* __restrict__ w, const float* __restrict__ beta,
                  const IO* __restrict__ r, const IO* __restrict__ k, const IO* __restrict__ v, float* state, IO* y,
                  bool vec) {
    // CL lanes of 4 value columns, 32 / CL lanes of R consecutive key rows
    constexpr int RG = 32 / CL, R = N / RG, CW = CL * 4, PARTS = N / CW;
    const int lane = threadIdx.x % 32;
    const int64_t id = int64_t(blockIdx.x) * NW + threadIdx.x / 32;
    pdl_begin();
    if (id >= heads * PARTS) return;
    const int64_t hh = id / PARTS;
    const int col = int(id % PARTS) * CW + (lane % CL) * 4, row = lane / CL * R;
    const int64_t hk = hh / H * Hk + hh % H / (H / Hk);
    float* sp = state + hh * N * N + row * N + col;
    float4 s[R];
    if (vec) {
#pragma unroll
        for (int i = 0; i < R; ++i) s[i] = __ldcs(reinterpret_cast<const float4*>(sp + i * N));
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) s[i] = make_float4(sp[i * N], sp[i * N + 1], sp[i * N + 2], sp[i * N + 3]);
    }
    const float a = expf(-w[hh]), bt = beta[hh];
    float kk[R];
#pragma unroll
    for (int i = 0; i < R; ++i) kk[i] = to_f32(k[hk * N + row + i]);
    float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        s[i].x *= a, s[i].y *= a, s[i].z *= a, s[i].w *= a;
        p.x = fmaf(s[i].x, kk[i], p.x);
        p.y = fmaf(s[i].y, kk[i], p.y);
        p.z = fmaf(s[i].z, kk[i], p.z);
        p.w = fmaf(s[i].w, kk[i], p.w);
    }
#pragma unroll
    for (int o = CL; o < 32; o *= 2) {
        p.x += __shfl_xor_sync(0xffffffffu, p.x, o);
        p.y += __shfl_xor_sync(0xffffffffu, p.y, o);
        p.z += __shfl_xor_sync(0xffffffffu, p.z, o);
        p.w += __shfl_xor_sync(0xffffffffu, p.w, o);
    }
    const IO* vp = v + hh * N + col;
    const float4 u = make_float4(bt * (to_f32(vp[0]) - p.x), bt * (to_f32(vp[1]) - p.y), bt * (to_f32(vp[2]) - p.z),
                                 bt * (to_f32(vp[3]) - p.w));
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float rr = to_f32(r[hk * N + row + i]);
        s[i].x = fmaf(kk[i], u.x, s[i].x);
        s[i].y = fmaf(kk[i], u.y, s[i].y);
        s[i].z = fmaf(kk[i], u.z, s[i].z);
        s[i].w = fmaf(kk[i], u.w, s[i].w);
        q.x = fmaf(s[i].x, rr, q.x);
        q.y = fmaf(s[i].y, rr, q.y);
        q.z = fmaf(s[i].z, rr, q.z);
        q.w = fmaf(s[i].w, rr, q.w);
    }
    if (vec) {
#pragma unroll
        for (int i = 0; i < R; ++i) __stcs(reinterpret_cast<float4*>(sp + i * N), s[i]);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) sp[i * N] = s[i].x, sp[i * N + 1] = s[i].y, sp[i * N + 2] = s[i].z, sp[i * N + 3] = s[i].w;
    }
#pragma unroll
    for (int o = CL; o < 32; o *= 2) {
        q.x += __shfl_xor_sync(0xffffffffu, q.x, o);
        q.y += __shfl_xor_sync(0xffffffffu, q.y, o);
        q.z += __shfl_xor_sync(0xffffffffu, q.z, o);
        q.w += __shfl_xor_sync(0xffffffffu, q.w, o);
    }
    if (lane < CL) {
        IO* yp = y + hh * N + col;
        put(yp, q.x), put(yp + 1, q.y), put(yp + 2, q.z), put(yp + 3, q.w);
    }
}

}  // namespace delta
}  // namespace wkv
