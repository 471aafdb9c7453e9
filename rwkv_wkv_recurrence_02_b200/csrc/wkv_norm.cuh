// wkv_norm.cuh -- group norm with an activation, channels last, forward and
// reverse: every token's channels in G groups (the heads of the matrix-state
// operators), each normalised by its own mean and variance.
//
//   hat = (x - mean) / sqrt(var + eps),  z = weight * hat + bias
//   y = act(z) without a gate, z * act(gate) with one
//
// A lane holds V vectors of PER channels of one group, LPG lanes a group (a
// power of two, the lanes behind the group's last channel idle), and keeps
// its channels over `span` tokens, so weight and bias stay in registers and
// the reverse mode sums dweight and dbias there.  Mean and variance are two
// passes over registers: x is read once.  Bound by memory, and near it by the
// instructions, so the arithmetic is in packed pairs.  8 x 4096 tokens of 2048
// bfloat16 channels in 32 groups with a gate: forward 80 us (5.0 TB/s, 78% of a
// copy's rate; 103 with loads into registers a token ahead instead of the ring),
// reverse 146 us (4.6 TB/s; 214).
#pragma once

#include "wkv_common.cuh"

namespace wkv {
namespace norm {

enum Act { kNone = 0, kSilu = 1, kSigmoid = 2 };

struct Args {
    int64_t rows, C;
    int group, lpg, lpg_log2;   // channels of a group, lanes of a group
    int64_t slots;              // lanes of a row, in whole warps
    int span;                   // rows a lane takes
    int act;
    float eps, inv_group;
    const void* x;
    const void* gate;
    const float* weight;
    const float* bias;
    const void* dy;
    void* y;
    void* dx;
    void* dgate;
    float* part;                // (chunks, 2, C) partial dweight, dbias or NULL
};

template <typename IO, int PER>
struct Pack {
    static_assert(PER * sizeof(IO) <= 16, "one access");
    static constexpr int WORDS = PER * int(sizeof(IO)) / 4 > 0 ? PER * int(sizeof(IO)) / 4 : 1;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const IO* p) {
        if constexpr (PER * sizeof(IO) == 16) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (PER * sizeof(IO) == 8) {
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (PER * sizeof(IO) == 4) {
            w[0] = __ldcs(reinterpret_cast<const unsigned int*>(p));
        } else {
            w[0] = __ldcs(reinterpret_cast<const unsigned short*>(p));
        }
    }
    __device__ __forceinline__ void load_shared(uint32_t addr) {
        if constexpr (PER * sizeof(IO) == 16)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
        else if constexpr (PER * sizeof(IO) == 8)
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
        else
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(IO) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    __device__ __forceinline__ void put(int i, float v) {
        if constexpr (sizeof(IO) == 4) {
            w[i] = __float_as_uint(v);
        } else {
            const uint32_t b = __bfloat16_as_ushort(__float2bfloat16_rn(v));
            if (i % 2) w[i / 2] |= b << 16;   // after the even one
            else w[i / 2] = b;
        }
    }
    __device__ __forceinline__ void store(IO* p) const {
        if constexpr (PER * sizeof(IO) == 16) __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
        else if constexpr (PER * sizeof(IO) == 8) __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
        else if constexpr (PER * sizeof(IO) == 4) __stcs(reinterpret_cast<unsigned int*>(p), w[0]);
        else *reinterpret_cast<unsigned short*>(p) = static_cast<unsigned short>(w[0]);
    }
};

// 1 / (1 + e^-x): ex2 and rcp are within 2 ulp, the argument's rounding adds
// |x| 2^-24 (the outputs' float32 bound is 2e-5)
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-x * kLog2e)); }
__device__ __forceinline__ float act(int kind, float x) {
    if (kind == kNone) return x;
    const float s = sigmoid(x);
    return kind == kSilu ? x * s : s;
}
// the activation and its slope
__device__ __forceinline__ float act_slope(int kind, float x, float* slope) {
    if (kind == kNone) {
        *slope = 1.f;
        return x;
    }
    const float s = sigmoid(x);
    if (kind == kSilu) {
        *slope = s * fmaf(x, 1.f - s, 1.f);
        return x * s;
    }
    *slope = s * (1.f - s);
    return s;
}

__device__ __forceinline__ float group_sum(float x, int lpg) {
    for (int o = lpg / 2; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// a lane's place: its group's first channel, the offsets of its vectors
template <int PER, int V>
struct Place {
    int64_t slot, chunk, c0;   // c0: the lane's first channel
    int n;                     // vectors of it that exist
    __device__ __forceinline__ Place(const Args& a) {
        const int64_t id = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
        slot = id % a.slots;
        chunk = id / a.slots;
        const int l = int(slot) & (a.lpg - 1);
        const int64_t grp = slot >> a.lpg_log2;
        c0 = grp * a.group + int64_t(l) * PER;
        const int vecs = a.group / PER;
        n = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (l + v * a.lpg < vecs) n = v + 1;
        if (grp * a.group >= a.C) n = 0;
    }
};

// Packed pairs of a lane's channels.  PER == 1 keeps one value a pair, the
// other half zero throughout.
template <int PER>
constexpr int kPairs = PER > 1 ? PER / 2 : 1;

template <typename IO, int PER>
__device__ __forceinline__ F2 pair_of(const Pack<IO, PER>& v, int i) {
    return f2(v.get(2 * i), PER > 1 ? v.get(2 * i + 1) : 0.f);
}
template <typename IO, int PER>
__device__ __forceinline__ void put_pair(Pack<IO, PER>& v, int i, F2 x) {
    if constexpr (PER > 1 && sizeof(IO) == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f2lo(x), f2hi(x));
        v.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
        v.put(2 * i, f2lo(x));
        if constexpr (PER > 1) v.put(2 * i + 1, f2hi(x));
    }
}
__device__ __forceinline__ F2 sigmoid2(F2 x) {
    const F2 e = ex2x2(mul2(x, f2s(-kLog2e)));
    return rcpx2(add2(e, f2s(1.f)));
}
__device__ __forceinline__ F2 neg2(F2 x) { return mul2(x, f2s(-1.f)); }

// weight and bias of a lane's channels
template <int PER, int V>
struct Affine {
    F2 w[V][kPairs<PER>], b[V][kPairs<PER>];
    __device__ __forceinline__ void load(const Args& a, const Place<PER, V>& at) {
        const int step = a.lpg * PER;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < kPairs<PER>; ++i) {
                float x[4] = {1.f, 1.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < (PER > 1 ? 2 : 1); ++q)
                    if (v < at.n) {
                        const int64_t c = at.c0 + v * step + 2 * i + q;
                        if (a.weight != nullptr) x[q] = __ldg(a.weight + c);
                        if (a.bias != nullptr) x[2 + q] = __ldg(a.bias + c);
                    }
                w[v][i] = f2(x[0], x[1]);
                b[v][i] = f2(x[2], x[3]);
            }
    }
};

// x - mean of a lane's channels (zero where there are none), and 1 / sqrt(var + eps)
template <typename IO, int PER, int V>
__device__ __forceinline__ float centre(const Args& a, const Place<PER, V>& at, const Pack<IO, PER> (&x)[V],
                                        F2 (&d)[V][kPairs<PER>]) {
    F2 s = f2s(0.f);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < kPairs<PER>; ++i) {
            d[v][i] = pair_of(x[v], i);
            s = add2(s, d[v][i]);
        }
    const float mean = group_sum(f2lo(s) + f2hi(s), a.lpg) * a.inv_group;
    s = f2s(0.f);
    const F2 m = PER > 1 ? f2s(-mean) : f2(-mean, 0.f);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < kPairs<PER>; ++i) {
            d[v][i] = v < at.n ? add2(d[v][i], m) : f2s(0.f);
            s = fma2(d[v][i], d[v][i], s);
        }
    return rsqrtf(fmaf(group_sum(f2lo(s) + f2hi(s), a.lpg), a.inv_group, a.eps));
}

// A lane's vectors of one token of each tensor
template <typename IO, int PER, int V, bool GATE, bool BWD>
struct Rows {
    Pack<IO, PER> x[V], gate[V], dy[V];
};

// The tokens a lane has on their way: a ring in shared memory that the lane
// fills and reads by itself (asynchronous copies, no barrier), STAGES - 1
// tokens ahead.  Registers would bound the bytes in flight, and with them the
// bandwidth.  Vectors of 2 bytes, which such copies cannot take, are read when
// they are needed.
template <typename IO, int PER, int V, bool GATE, bool BWD>
struct Ring {
    static constexpr int B = PER * int(sizeof(IO)), NT = 1 + GATE + BWD;
    static constexpr bool ASYNC = B >= 4;
    static constexpr int STAGE = NT * V * B * 256;
    static constexpr int FIT = 48 * 1024 / STAGE;
    static constexpr int STAGES = !ASYNC ? 1 : FIT > 5 ? 5 : FIT < 2 ? 2 : FIT;
    static constexpr int SMEM = ASYNC ? STAGES * STAGE : 0;
    uint32_t base;
    int fill, take;
    __device__ __forceinline__ Ring() : fill(0), take(0) {
        extern __shared__ __align__(16) char smem[];
        base = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + threadIdx.x * B;
    }
    // token r's copies (none behind the last: an empty group keeps the count)
    __device__ __forceinline__ void ask(const Args& a, const Place<PER, V>& at, int64_t r, int64_t r1) {
        if constexpr (ASYNC) {
            if (r < r1) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v < at.n) {
                        const int64_t off = r * a.C + at.c0 + v * (a.lpg * PER);
                        const uint32_t dst = base + fill * STAGE + v * B * 256;
                        copy(dst, static_cast<const IO*>(a.x) + off);
                        if constexpr (BWD) copy(dst + V * B * 256, static_cast<const IO*>(a.dy) + off);
                        if constexpr (GATE) copy(dst + (1 + BWD) * V * B * 256, static_cast<const IO*>(a.gate) + off);
                    }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            fill = fill + 1 == STAGES ? 0 : fill + 1;
        }
    }
    static __device__ __forceinline__ void copy(uint32_t dst, const void* src) {
        if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(B >= 4 ? B : 4) : "memory");
    }
    // the oldest token asked for (token r)
    __device__ __forceinline__ void get(const Args& a, const Place<PER, V>& at, int64_t r, Rows<IO, PER, V, GATE, BWD>& t) {
        if constexpr (ASYNC) asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
#pragma unroll
        for (int v = 0; v < V; ++v) {
            t.x[v].clear();
            if (BWD) t.dy[v].clear();
            if (GATE) t.gate[v].clear();
            if (v < at.n) {
                if constexpr (ASYNC) {
                    const uint32_t src = base + take * STAGE + v * B * 256;
                    t.x[v].load_shared(src);
                    if constexpr (BWD) t.dy[v].load_shared(src + V * B * 256);
                    if constexpr (GATE) t.gate[v].load_shared(src + (1 + BWD) * V * B * 256);
                } else {
                    const int64_t off = r * a.C + at.c0 + v * (a.lpg * PER);
                    t.x[v].load(static_cast<const IO*>(a.x) + off);
                    if constexpr (BWD) t.dy[v].load(static_cast<const IO*>(a.dy) + off);
                    if constexpr (GATE) t.gate[v].load(static_cast<const IO*>(a.gate) + off);
                }
            }
        }
        take = take + 1 == STAGES ? 0 : take + 1;
    }
};

template <typename IO, int PER, int V, bool GATE>
__device__ __forceinline__ void forward_row(const Args& a, const Place<PER, V>& at, const Affine<PER, V>& p,
                                            const Rows<IO, PER, V, GATE, false>& t, int64_t r) {
    F2 d[V][kPairs<PER>];
    const F2 inv = f2s(centre<IO, PER, V>(a, at, t.x, d));
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (v >= at.n) continue;
        Pack<IO, PER> o;
#pragma unroll
        for (int i = 0; i < kPairs<PER>; ++i) {
            const F2 z = fma2(mul2(d[v][i], inv), p.w[v][i], p.b[v][i]);
            F2 g = GATE ? pair_of(t.gate[v], i) : z;
            if (a.act != kNone) {
                const F2 s = sigmoid2(g);
                g = a.act == kSilu ? mul2(g, s) : s;
            }
            put_pair(o, i, GATE ? mul2(z, g) : g);
        }
        o.store(static_cast<IO*>(a.y) + r * a.C + at.c0 + v * (a.lpg * PER));
    }
}

template <typename IO, int PER, int V, bool GATE>
__global__ void __launch_bounds__(256, PER * V <= 8 ? 5 : 2) forward_kernel(const Args a) {
    pdl_begin();
    const Place<PER, V> at(a);
    const int64_t r0 = at.chunk * a.span;
    if (r0 >= a.rows) return;   // whole warps: slots is a multiple of 32
    const int64_t r1 = r0 + a.span < a.rows ? r0 + a.span : a.rows;
    using R = Ring<IO, PER, V, GATE, false>;
    R ring;
#pragma unroll
    for (int i = 0; i < R::STAGES - 1; ++i) ring.ask(a, at, r0 + i, r1);
    Affine<PER, V> p;
    p.load(a, at);
#pragma unroll 1
    for (int64_t r = r0; r < r1; ++r) {
        Rows<IO, PER, V, GATE, false> t;
        ring.get(a, at, r, t);
        ring.ask(a, at, r + R::STAGES - 1, r1);   // into the place of the token before this one
        forward_row<IO, PER, V, GATE>(a, at, p, t, r);
    }
}

// dz = dy act'(z) without a gate, dy act(gate) with one (dgate = dy z act'(gate));
// dweight = sum dz hat, dbias = sum dz over the tokens;
// dx = (h - mean(h) - hat mean(h hat)) / sqrt(var + eps), h = weight dz.
template <typename IO, int PER, int V, bool GATE, int ACT>
__device__ __forceinline__ void backward_row(const Args& a, const Place<PER, V>& at, const Affine<PER, V>& p,
                                             const Rows<IO, PER, V, GATE, true>& t, int64_t r, F2 (&dw)[V][kPairs<PER>],
                                             F2 (&db)[V][kPairs<PER>]) {
    constexpr int P = kPairs<PER>;
    F2 hat[V][P], h[V][P];
    const float inv = centre<IO, PER, V>(a, at, t.x, hat);
    F2 h1 = f2s(0.f), h2 = f2s(0.f);
    const int64_t row = r * a.C + at.c0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        Pack<IO, PER> o;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            hat[v][i] = mul2(hat[v][i], f2s(inv));
            const F2 z = fma2(hat[v][i], p.w[v][i], p.b[v][i]);
            const F2 g = GATE ? pair_of(t.gate[v], i) : z, dy = pair_of(t.dy[v], i);
            F2 value = g, slope = f2s(1.f);
            if (ACT != kNone) {
                const F2 s = sigmoid2(g), rest = fma2(s, f2s(-1.f), f2s(1.f));   // 1 - s
                value = ACT == kSilu ? mul2(g, s) : s;
                slope = mul2(s, ACT == kSilu ? fma2(g, rest, f2s(1.f)) : rest);
            }
            const F2 dz = mul2(dy, GATE ? value : slope);
            if constexpr (GATE) put_pair(o, i, mul2(mul2(dy, z), slope));
            dw[v][i] = fma2(dz, hat[v][i], dw[v][i]);
            db[v][i] = add2(db[v][i], dz);
            h[v][i] = mul2(p.w[v][i], dz);
            h1 = add2(h1, h[v][i]);
            h2 = fma2(h[v][i], hat[v][i], h2);
        }
        if (GATE && v < at.n) o.store(static_cast<IO*>(a.dgate) + row + v * (a.lpg * PER));
    }
    const float m1 = group_sum(f2lo(h1) + f2hi(h1), a.lpg) * a.inv_group;
    const float m2 = group_sum(f2lo(h2) + f2hi(h2), a.lpg) * a.inv_group;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (v >= at.n) continue;
        Pack<IO, PER> o;
#pragma unroll
        for (int i = 0; i < P; ++i)
            put_pair(o, i, mul2(fma2(hat[v][i], f2s(-m2), add2(h[v][i], f2s(-m1))), f2s(inv)));
        o.store(static_cast<IO*>(a.dx) + row + v * (a.lpg * PER));
    }
}

// ACT known to the compiler: a test of it at every pair took an eighth of the time
template <typename IO, int PER, int V, bool GATE, int ACT>
__global__ void __launch_bounds__(256, PER * V <= 8 ? 2 : 1) backward_kernel(const Args a) {
    pdl_begin();
    constexpr int P = kPairs<PER>;
    const Place<PER, V> at(a);
    const int64_t r0 = at.chunk * a.span;
    if (r0 >= a.rows) return;
    const int64_t r1 = r0 + a.span < a.rows ? r0 + a.span : a.rows;
    using R = Ring<IO, PER, V, GATE, true>;
    R ring;
#pragma unroll
    for (int i = 0; i < R::STAGES - 1; ++i) ring.ask(a, at, r0 + i, r1);
    Affine<PER, V> p;
    p.load(a, at);
    F2 dw[V][P], db[V][P];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < P; ++i) dw[v][i] = db[v][i] = f2s(0.f);
#pragma unroll 1
    for (int64_t r = r0; r < r1; ++r) {
        Rows<IO, PER, V, GATE, true> t;
        ring.get(a, at, r, t);
        ring.ask(a, at, r + R::STAGES - 1, r1);
        backward_row<IO, PER, V, GATE, ACT>(a, at, p, t, r, dw, db);
    }
    if (a.part != nullptr) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < at.n)
#pragma unroll
                for (int i = 0; i < P; ++i)
#pragma unroll
                    for (int q = 0; q < (PER > 1 ? 2 : 1); ++q) {
                        const int64_t c = at.c0 + v * (a.lpg * PER) + 2 * i + q;
                        a.part[(at.chunk * 2) * a.C + c] = q ? f2hi(dw[v][i]) : f2lo(dw[v][i]);
                        a.part[(at.chunk * 2 + 1) * a.C + c] = q ? f2hi(db[v][i]) : f2lo(db[v][i]);
                    }
    }
}

// Groups too large for registers: one CTA per (token, group), the group read
// again from the caches for each pass.
__device__ __forceinline__ float block_sum(float x, float* sm) {
    for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sm[threadIdx.x / 32] = x;
    __syncthreads();
    x = 0.f;
    for (int i = 0; i < int(blockDim.x) / 32; ++i) x += sm[i];
    return x;
}

template <typename IO>
__device__ __forceinline__ float at1(const void* p, int64_t i) {
    if constexpr (sizeof(IO) == 4) return static_cast<const float*>(p)[i];
    else return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <typename IO>
__device__ __forceinline__ void put1(void* p, int64_t i, float v) {
    if constexpr (sizeof(IO) == 4) static_cast<float*>(p)[i] = v;
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

template <typename IO, bool BWD>
__global__ void __launch_bounds__(256) large_kernel(const Args a, int64_t groups) {
    __shared__ float sm[8];
    pdl_begin();
    for (int64_t id = blockIdx.x; id < a.rows * groups; id += gridDim.x) {
        const int64_t r = id / groups, base = (id % groups) * a.group;
        const int64_t off = r * a.C + base;
        float s = 0.f;
        for (int i = threadIdx.x; i < a.group; i += blockDim.x) s += at1<IO>(a.x, off + i);
        const float mean = block_sum(s, sm) * a.inv_group;
        s = 0.f;
        for (int i = threadIdx.x; i < a.group; i += blockDim.x) {
            const float d = at1<IO>(a.x, off + i) - mean;
            s = fmaf(d, d, s);
        }
        const float inv = rsqrtf(fmaf(block_sum(s, sm), a.inv_group, a.eps));
        float h1 = 0.f, h2 = 0.f;
        for (int pass = 0; pass < (BWD ? 2 : 1); ++pass) {
            for (int i = threadIdx.x; i < a.group; i += blockDim.x) {
                const float wt = a.weight ? a.weight[base + i] : 1.f, bs = a.bias ? a.bias[base + i] : 0.f;
                const float hat = (at1<IO>(a.x, off + i) - mean) * inv, z = fmaf(hat, wt, bs);
                if constexpr (!BWD) {
                    put1<IO>(a.y, off + i, a.gate ? z * act(a.act, at1<IO>(a.gate, off + i)) : act(a.act, z));
                } else {
                    const float g = at1<IO>(a.dy, off + i);
                    float slope, dz;
                    if (a.gate) {
                        dz = g * act_slope(a.act, at1<IO>(a.gate, off + i), &slope);
                        if (pass == 0) put1<IO>(a.dgate, off + i, g * z * slope);
                    } else {
                        act_slope(a.act, z, &slope);
                        dz = g * slope;
                    }
                    const float h = wt * dz;
                    if (pass == 0) {
                        h1 += h;
                        h2 = fmaf(h, hat, h2);
                    } else {
                        put1<IO>(a.dx, off + i, inv * (h - h1 - hat * h2));
                    }
                }
            }
            if (BWD && pass == 0) {
                h1 = block_sum(h1, sm) * a.inv_group;
                h2 = block_sum(h2, sm) * a.inv_group;
            }
        }
        if constexpr (BWD) {
            // per (token, group) statistics for the parameters' sums
            if (threadIdx.x == 0 && a.part != nullptr) a.part[2 * id] = mean, a.part[2 * id + 1] = inv;
        }
    }
}

// dweight, dbias of large groups: each thread one channel over a chunk of
// tokens, with the statistics that large_kernel left.
template <typename IO>
__global__ void __launch_bounds__(128) large_params_kernel(const Args a, int64_t groups, const float* __restrict__ stats,
                                                           float* __restrict__ part, int64_t per) {
    const int64_t c = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    pdl_begin();
    if (c >= a.C) return;
    const float wt = a.weight ? a.weight[c] : 1.f, bs = a.bias ? a.bias[c] : 0.f;
    const int64_t r0 = blockIdx.y * per, r1 = r0 + per < a.rows ? r0 + per : a.rows, grp = c / a.group;
    float dw = 0.f, db = 0.f;
    for (int64_t r = r0; r < r1; ++r) {
        const float2 st = reinterpret_cast<const float2*>(stats)[r * groups + grp];
        const float hat = (at1<IO>(a.x, r * a.C + c) - st.x) * st.y;
        float slope, dz = at1<IO>(a.dy, r * a.C + c);
        if (a.gate) {
            dz *= act(a.act, at1<IO>(a.gate, r * a.C + c));
        } else {
            act_slope(a.act, fmaf(hat, wt, bs), &slope);
            dz *= slope;
        }
        dw = fmaf(dz, hat, dw);
        db += dz;
    }
    part[(int64_t(blockIdx.y) * 2) * a.C + c] = dw;
    part[(int64_t(blockIdx.y) * 2 + 1) * a.C + c] = db;
}

// the chunks' partial sums, in a fixed order: 32 channels x 32 warps of chunks
__global__ void __launch_bounds__(1024) params_kernel(int64_t C, int64_t chunks, const float* __restrict__ part,
                                                      float* __restrict__ dweight, float* __restrict__ dbias) {
    __shared__ float sm[2][32][33];
    const int cx = threadIdx.x % 32, k = threadIdx.x / 32;
    const int64_t c = int64_t(blockIdx.x) * 32 + cx;
    pdl_begin();
    float dw = 0.f, db = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int64_t i = k; i < chunks; i += 32) {
            dw += part[2 * i * C + c];
            db += part[(2 * i + 1) * C + c];
        }
    }
    sm[0][k][cx] = dw;
    sm[1][k][cx] = db;
    __syncthreads();
    // warp k: the sums of channel k
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        float s = sm[o][cx][k];
#pragma unroll
        for (int w = 16; w > 0; w /= 2) s += __shfl_xor_sync(0xffffffffu, s, w);
        float* out = o == 0 ? dweight : dbias;
        const int64_t ch = int64_t(blockIdx.x) * 32 + k;
        if (cx == 0 && out != nullptr && ch < C) out[ch] = s;
    }
}

}  // namespace norm
}  // namespace wkv
