// wkv_delta_mma.cuh -- the gated delta rule in chunks of 16 tokens on the
// tensor cores, with the state at float32 accuracy.
//
// Within a chunk that enters with state S, G[t][s] the product of the decays
// of tokens s+1 .. t and g_t that of tokens 0 .. t:
//   (I + A) E = V - diag(g) K S,       A[t][s] = G[t][s] beta_s k_t.k_s  (s < t)
//   Y  = diag(g) R S + P E,            P[t][s] = G[t][s] beta_s r_t.k_s  (s <= t)
//   S <- g_15 S + K^T diag(G[15][.] beta) E
// No decay is divided by, so resets and strong decays need no case of their
// own.
//
// A warp keeps S^T for 16 value columns and the whole key axis as mma
// accumulators (m = value, n = key).  The accumulator layout of one product is
// the A-operand layout of the next, so S^T -> K S -> E -> S^T stays in
// registers and the walking warps exchange nothing; K, R and V come from shared
// memory by ldmatrix.  A, its inverse and P do not depend on the state: staging
// warps, one for each of four stages, fetch a chunk and form them chunks
// ahead.
//
// Accuracy: a float32 operand is the sum of three bfloat16 pieces (24 bits);
// products of pieces up to 2^-16 of the leading one are taken, the leading one
// in an accumulator of its own.  bfloat16 inputs are one piece, exact: three
// products with a float32 operand.  So a bfloat16 output is a float32 sum rounded
// once.  The state is updated by a float32 multiply-add of the chunk's sum, so
// the accumulators' truncation does not add up along T.
//
// Values that are not finite: the zeros of these matrices, times a NaN, would carry
// it to the tokens ahead of its own.  It always reaches the column's state, and
// stays there.  So a walk that ends with a column not finite which began finite is
// walked again, token by token (forward_again; 8 x 4096 tokens of 32 heads of 64 then
// take 1765 us).  A test of every chunk's E in the first place, or only the code for it
// in the loop, took 6% of the time of all calls.
//
// What bounds it: issue.  An mma.sync of 16 x 8 x 16 holds its scheduler for 8.3
// cycles here and other instructions do not issue meanwhile; bfloat16 heads of 64
// have 96 of the ones and about 500 of the others a chunk and warp.  On an SM with
// two walks the tensor pipe is active in 51% of the cycles and an instruction
// issues in 44%.  Measured: 8 x 4096 tokens
// of 32 heads of 64 in bfloat16 429 us (reads and writes alone: 85; the same
// recurrence token by token in float32 multiply-adds: 1798).  With few heads a
// chunk's chain of dependent products bounds it: 32 heads x 4096 tokens 242 us
// (0.95 us a chunk), 32 heads of 128 395 us.  Chunks of 32 tokens were no faster
// (the code outgrows the instruction cache), 2 or 4 warps sharing a head's keys
// slower (583 us against 386, exchange in shared memory), fp16 pieces slower (428 us
// against 402, the scaling).
#pragma once

#include "wkv_delta.cuh"

namespace wkv {
namespace delta {

constexpr int kChunk = 16;     // tokens of a chunk: one k step of an mma
constexpr int kMat = kChunk * kChunk;
// Place of (row, column) in a 16 x 16 bfloat16 matrix: the two halves of rows
// 4 .. 7 (mod 8) change places, so that eight rows of ldmatrix differ in banks.
__device__ __forceinline__ int mat_at(int r, int c) { return r * kChunk + (((c >> 3) ^ (r >> 2)) & 1) * 8 + (c & 7); }

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void stsm2t(uint32_t addr, const uint32_t (&r)[2]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1,%2};" :: "r"(addr), "r"(r[0]), "r"(r[1]) : "memory");
}
// a 16 x 16 accumulator as bfloat16, rows as they lie
__device__ __forceinline__ void stsm_tile(uint32_t addr, const float (&c)[2][4]) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(c[i / 2][i % 2 * 2], c[i / 2][i % 2 * 2 + 1]);
        r[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
// c += A B, or c = A B
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// a 16-wide B operand (two tiles)
__device__ __forceinline__ void mma2(float (&c)[2][4], const uint32_t (&a)[4], const uint32_t (&f)[4], bool first) {
    if (first) {
        mma_first(c[0], a, f[0], f[1]);
        mma_first(c[1], a, f[2], f[3]);
    } else {
        mma(c[0], a, f[0], f[1]);
        mma(c[1], a, f[2], f[3]);
    }
}
// barriers of the staging warps and the walking warps
template <int THREADS>
__device__ __forceinline__ void bar_sync(int id) { asm volatile("bar.sync %0, %1;" :: "r"(id), "n"(THREADS) : "memory"); }
template <int THREADS>
__device__ __forceinline__ void bar_arrive(int id) { asm volatile("bar.arrive %0, %1;" :: "r"(id), "n"(THREADS) : "memory"); }
// all of them: does p hold for one?
template <int THREADS>
__device__ __forceinline__ bool bar_or(int id, bool p) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(uint32_t(p)), "r"(id), "n"(THREADS) : "memory");
    return r != 0;
}
// ids: one for each of four stages
constexpr int kBarFull = 1, kBarFree = 5, kBarTask = 9;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" :: "l"(p)); }

// (x, y) as NP packed bfloat16 pairs whose sum is the pair to 8 NP bits
template <int NP>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&p)[NP]) {
    F2 v = f2(x, y);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f2lo(v), f2hi(v));
        p[i] = *reinterpret_cast<const uint32_t*>(&h);
        if (i + 1 < NP) v = fma2(f2(__uint_as_float(p[i] << 16), __uint_as_float(p[i] & 0xffff0000u)), f2s(-1.f), v);
    }
}
// Two neighbouring accumulator tiles (16 x 16) as the pieces of an A operand
template <int NP>
__device__ __forceinline__ void split_a(const float (&c0)[4], const float (&c1)[4], uint32_t (&a)[NP][4]) {
    uint32_t p[NP];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float* c = q < 2 ? c0 : c1;
        split2<NP>(c[(q & 1) * 2], c[(q & 1) * 2 + 1], p);
#pragma unroll
        for (int i = 0; i < NP; ++i) a[i][q] = p[i];
    }
}

// A float2 of a token pair's factors: tokens 8 n + 2 (lane % 4) + {0, 1}
__device__ __forceinline__ float2 pair_at(const float* x, int n, int lane) {
    return *reinterpret_cast<const float2*>(x + 8 * n + 2 * (lane % 4));
}

// Places of (row, column) in shared memory: rows of LD elements, or (Swizzled)
// of W without padding, 16-byte pieces in an order of their own in every row, so
// that eight rows of ldmatrix differ in banks.
template <int LD>
struct Pitched {
    __device__ __forceinline__ int operator()(int r, int c) const { return r * LD + c; }
};
template <int W>
struct Swizzled {
    static __device__ __forceinline__ int turn(int r) { return W == 32 ? (r >> 1) & 3 : r & 7; }
    __device__ __forceinline__ int operator()(int r, int c) const { return r * W + (((c >> 3) ^ turn(r)) << 3) + (c & 7); }
};
// One warp's copy of ROWS rows of W elements to shared memory: 16-byte
// asynchronous copies, or element copies where the addresses do not
// allow them; rows from nt on are zero.
template <typename IO, int ROWS, int W, typename AT>
__device__ __forceinline__ void copy_rows(IO* dst, AT at, const IO* src, int64_t stride, int nt, bool vec, int lane) {
    if (vec) {
        constexpr int PER = 16 / int(sizeof(IO)), ROWV = W / PER;
#pragma unroll
        for (int i = lane; i < ROWS * ROWV; i += 32) {
            const int t = i / ROWV, c = (i % ROWV) * PER;
            cp_async16(smem_u32(dst + at(t, c)), src + (t < nt ? t : 0) * stride + c, t < nt);
        }
    } else {
        for (int i = lane; i < ROWS * W; i += 32) {
            const int t = i / W, c = i % W;
            IO x;
            if constexpr (sizeof(IO) == 4) x = 0.f;
            else x = __ushort_as_bfloat16(0);
            if (t < nt) x = src[t * stride + c];
            dst[at(t, c)] = x;
        }
    }
}

__device__ __forceinline__ float4 load4(const float* p, bool vec) {
    return vec ? __ldcg(reinterpret_cast<const float4*>(p)) : make_float4(p[0], p[1], p[2], p[3]);
}
// four neighbouring values as NP bfloat16 pieces, `piece` elements apart
template <int NP>
__device__ __forceinline__ void put4(__nv_bfloat16* dst, int piece, float4 v) {
    uint32_t p[NP], q[NP];
    split2<NP>(v.x, v.y, p);
    split2<NP>(v.z, v.w, q);
#pragma unroll
    for (int i = 0; i < NP; ++i) *reinterpret_cast<uint2*>(dst + i * piece) = make_uint2(p[i], q[i]);
}
// One warp's copy of ROWS float32 rows as NP arrays of pieces, rows from nt on
// as zeros (src itself is a row that exists)
template <int ROWS, int W, int NP, typename AT>
__device__ __forceinline__ void split_rows(__nv_bfloat16* dst, AT at, int piece, const float* src, int64_t stride, int nt, bool vec,
                                           int lane) {
    constexpr int ROWV = W / 4, ALL = ROWS * ROWV / 32, U = ALL < 8 ? ALL : 8;   // U loads in flight
#pragma unroll 1
    for (int n = 0; n < ALL; n += U) {
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = lane + (n + u) * 32, t = i / ROWV, c = (i % ROWV) * 4;
            v[u] = load4(src + (t < nt ? t : 0) * stride + c, vec);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = lane + (n + u) * 32, t = i / ROWV, c = (i % ROWV) * 4;
            if (t >= nt) v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            put4<NP>(dst + at(t, c), piece, v[u]);
        }
    }
}

// Column j = lane % 16 of (I + A)^-1, A strictly lower triangular 16 x 16 in
// shared memory (row pitch 20), by forward substitution.
__device__ __forceinline__ void invert_column(const float* A, int lane, float (&x)[kChunk]) {
    const int j = lane % 16;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        float acc[2] = {i == j ? 1.f : 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < i; m += 4) {
            const float4 a = *reinterpret_cast<const float4*>(A + i * 20 + m);
            const float e[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (m + q < i) acc[q & 1] = fmaf(-e[q], x[m + q], acc[q & 1]);
        }
        x[i] = acc[0] + acc[1];
    }
}

// Decays of NTOK tokens (one warp; a lane is a token).  The running sum W of the
// rates goes to shared memory as two float32 (its 64-bit value to 48 bits), so
// that W_t - W_s is as exact as a float32 however far in the two tokens lie.
// e^-kMaxRate is 0.
constexpr float kMaxRate = 1e4f;
struct ChunkDecay {
    float upto, after;   // the products of the decays up to a token, and after it
};
__device__ __forceinline__ float decay_of(float2 t, float2 s) { return ex2(-kLog2e * ((t.x - s.x) + (t.y - s.y))); }
__device__ __forceinline__ float2 two_floats(double x) {
    const float a = float(x);
    return make_float2(a, float(x - double(a)));
}
template <int NTOK>
__device__ __forceinline__ ChunkDecay chunk_decay(float w, float2* sums, int lane) {
    double x = w > kMaxRate ? kMaxRate : w;
#pragma unroll
    for (int o = 1; o < NTOK; o *= 2) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    const float2 v = two_floats(x);
    if (lane < NTOK) sums[lane] = v;
    const float2 last = make_float2(__shfl_sync(0xffffffffu, v.x, NTOK - 1), __shfl_sync(0xffffffffu, v.y, NTOK - 1));
    return ChunkDecay{decay_of(v, make_float2(0.f, 0.f)), decay_of(last, v)};
}

// (v0, v1) of row t, columns s, s + 1 into the pieces of a 16 x 16 matrix
template <int NP>
__device__ __forceinline__ void put_pieces(__nv_bfloat16* m, int t, int s, float v0, float v1) {
    uint32_t p[NP];
    split2<NP>(v0, v1, p);
#pragma unroll
    for (int q = 0; q < NP; ++q) *reinterpret_cast<uint32_t*>(m + q * kMat + mat_at(t, s)) = p[q];
}

// The inverse of I + A (A in shared memory) as three pieces.
__device__ __forceinline__ void put_inverse(__nv_bfloat16* m, const float* A, int lane) {
    float x[kChunk];
    invert_column(A, lane, x);
#pragma unroll
    for (int i = 0; i < kChunk / 2; ++i) {
        const float v = lane < 16 ? x[i] : x[i + 8];
        const int t = lane < 16 ? i : i + 8;
        uint32_t p[3];
        split2<3>(v, 0.f, p);
#pragma unroll
        for (int q = 0; q < 3; ++q) m[q * kMat + mat_at(t, lane % 16)] = __ushort_as_bfloat16(static_cast<unsigned short>(p[q]));
    }
}

// shared-memory offsets (elements) of this lane in a B operand: rows as they
// lie (row = column of the product) and transposed (row = its k)
__device__ __forceinline__ int b_plain(int lane, int ld) { return ((lane & 7) + (lane >> 4) * 8) * ld + ((lane >> 3) & 1) * 8; }
__device__ __forceinline__ int b_trans(int lane, int ld) { return ((lane & 7) + ((lane >> 3) & 1) * 8) * ld + (lane >> 4) * 8; }
// and in a 16 x 16 matrix
__device__ __forceinline__ int m_plain(int lane) { return mat_at((lane & 7) + (lane >> 4) * 8, ((lane >> 3) & 1) * 8); }
__device__ __forceinline__ int m_trans(int lane) { return mat_at((lane & 7) + ((lane >> 3) & 1) * 8, (lane >> 4) * 8); }

// A 16-token x 16-line tile of staged rows, transposed, in the accumulator
// layout: x[n][i] is line lane / 4 + 8 (i / 2), token 8 n + 2 (lane % 4) + i % 2.
template <typename IO>
__device__ __forceinline__ void load_lines(float (&x)[2][4], const IO* rows, int ld, int lane) {
    if constexpr (sizeof(IO) == 2) {
        uint32_t f[4];
        const int m = lane >> 3;
        ldsm4t(f, smem_u32(rows + ((lane & 7) + (m >> 1) * 8) * ld + (m & 1) * 8));
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[n][i] = __uint_as_float((i & 1) ? f[2 * n + (i >> 1)] & 0xffff0000u : f[2 * n + (i >> 1)] << 16);
    } else {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[n][i] = to_f32(rows[(8 * n + 2 * (lane % 4) + (i & 1)) * ld + lane / 4 + (i >> 1) * 8]);
    }
}

// One of its 8-token halves to rows of global memory (row t at out + t *
// stride), rows below nt.  bfloat16 goes through `rows`, a place of eight
// staged rows of its own, to 16-byte stores.
template <typename OUT, typename IO>
__device__ __forceinline__ void store_half(OUT* out, int64_t stride, int nt, const float (&x)[4], IO* rows, int ld, bool vec,
                                           int lane) {
    if constexpr (sizeof(OUT) == 2) {
        uint32_t f[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const __nv_bfloat162 v2 = __floats2bfloat162_rn(x[2 * q], x[2 * q + 1]);
            f[q] = *reinterpret_cast<const uint32_t*>(&v2);
        }
        stsm2t(smem_u32(rows + (lane & 7) * ld + ((lane >> 3) & 1) * 8), f);
        __syncwarp();
        const int t = (lane / 2) % 8, col = (lane % 2) * 8;
        const uint4 v4 = *reinterpret_cast<const uint4*>(rows + t * ld + col);
        if (lane < 16 && t < nt) {
            OUT* o = out + t * stride + col;
            if (vec) {
                *reinterpret_cast<uint4*>(o) = v4;
            } else {
                const uint32_t wd[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    reinterpret_cast<unsigned short*>(o)[i] = static_cast<unsigned short>(wd[i / 2] >> (16 * (i & 1)));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 2 * (lane % 4) + (i & 1);
            if (t < nt) out[t * stride + lane / 4 + (i >> 1) * 8] = x[i];
        }
    }
}

// x times a factor for each token
__device__ __forceinline__ void scale_tokens(float (&x)[2][4], const float* f, int lane) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const float2 v = pair_at(f, n, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] *= (i & 1) ? v.y : v.x;
    }
}

// A product of pieces in two accumulators: the leading order, and all others
// (2^-8 of it, so what their additions cut off is 2^-8 of a float32 step).  The
// leading one is added to a float32 sum every CHAIN steps of 16: the tensor
// cores cut off what a rounded addition would keep half of, so errors of a long
// chain have one sign and grow with its length.
struct Acc {
    float hi[2][4], lo[2][4];
    // before k step kk: does the leading order begin anew?  x: the sum of the steps before
    template <int CHAIN>
    __device__ __forceinline__ bool start(float (&x)[2][4], int kk) const {
        if (kk > 0 && kk % CHAIN == 0) add(x, hi, kk == CHAIN);
        return kk % CHAIN == 0;
    }
    // after the last of `steps`
    template <int CHAIN>
    __device__ __forceinline__ void finish(float (&x)[2][4], int steps, bool has_lo = true) const {
        add(x, hi, steps <= CHAIN);
        if (has_lo) add(x, lo, false);
    }
    __device__ __forceinline__ void sum(float (&x)[2][4]) const { finish<1>(x, 1); }
    static __device__ __forceinline__ void add(float (&x)[2][4], const float (&y)[2][4], bool first) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const F2 v = first ? f2(y[n][i], y[n][i + 1]) : add2(f2(x[n][i], x[n][i + 1]), f2(y[n][i], y[n][i + 1]));
                x[n][i] = f2lo(v), x[n][i + 1] = f2hi(v);
            }
    }
};
// (16 tokens x N) (N x 16 tokens)^T of two staged arrays of KX and KY pieces
// (`piece` bytes apart), the products of the first ORD orders: C[t][s] = x_t .
// y_s.  xa, ya: this lane's place in the first 16 columns of x as an A operand,
// of y as a plain B operand; SWIZZLED: the columns' places by exclusive or.
template <int N, int KX, int KY, int ORD, int CHAIN, bool SWIZZLED>
__device__ __forceinline__ void gram_at(float (&c)[2][4], uint32_t xa, uint32_t ya, int piece) {
    Acc acc;
#pragma unroll
    for (int kk = 0; kk < N / 16; ++kk) {
        uint32_t a[KX][4], b[KY][4];
#pragma unroll
        for (int p = 0; p < KX; ++p) ldsm4(a[p], (SWIZZLED ? xa ^ (kk * 32) : xa + kk * 32) + p * piece);
#pragma unroll
        for (int p = 0; p < KY; ++p) ldsm4(b[p], (SWIZZLED ? ya ^ (kk * 32) : ya + kk * 32) + p * piece);
        const bool hi_first = acc.start<CHAIN>(c, kk);
        bool lo_first = kk == 0;
#pragma unroll
        for (int p = 0; p < KX && p < ORD; ++p)
#pragma unroll
            for (int q = 0; q < KY && p + q < ORD; ++q) {
                mma2(p + q == 0 ? acc.hi : acc.lo, a[p], b[q], p + q == 0 ? hi_first : lo_first);
                if (p + q > 0) lo_first = false;
            }
    }
    acc.finish<CHAIN>(c, N / 16, ORD > 1 && KX * KY > 1);
}
template <int N, int KX, int KY, int ORD, int CHAIN>
__device__ __forceinline__ void gram(float (&c)[2][4], const __nv_bfloat16* x, const __nv_bfloat16* y, int piece, int lane) {
    constexpr int LD = N + 8;
    gram_at<N, KX, KY, ORD, CHAIN, false>(c, smem_u32(x + b_trans(lane, LD)), smem_u32(y + b_plain(lane, LD)), piece * 2);
}

// acc (+)= A (16 x 16) B (16 x 16) of NA and NB pieces, orders below ORD.  B's
// pieces lie `piece` elements apart, off: this lane's offset (b_plain, b_trans)
template <int NA, int NB, int ORD, bool TRANS>
__device__ __forceinline__ void times(Acc& acc, bool first, bool lo_first, const uint32_t (&a)[NA][4], const __nv_bfloat16* m,
                                      int piece, int off) {
    const uint32_t addr = smem_u32(m + off);
#pragma unroll
    for (int p = 0; p < NB && p < ORD; ++p) {
        uint32_t f[4];
        if constexpr (TRANS) ldsm4t(f, addr + p * piece * 2);
        else ldsm4(f, addr + p * piece * 2);
#pragma unroll
        for (int i = 0; i < NA && i + p < ORD; ++i) {
            mma2(i + p == 0 ? acc.hi : acc.lo, a[i], f, i + p == 0 ? first : lo_first);
            if (i + p > 0) lo_first = false;
        }
    }
}
// d (+)= A B into one accumulator, smallest orders first
template <int NA, int NB, int ORD>
__device__ __forceinline__ void times_sum(float (&d)[2][4], bool first, const uint32_t (&a)[NA][4], const uint32_t (&f)[NB][4]) {
#pragma unroll
    for (int o = ORD - 1; o >= 0; --o)
#pragma unroll
        for (int p = 0; p < NB && p <= o; ++p)
            if (o - p < NA) {
                mma2(d, a[o - p], f[p], first);
                first = false;
            }
}
template <int NA, int NB>
__device__ __forceinline__ void times_add(float (&d)[2][4], bool first, const uint32_t (&a)[NA][4], const __nv_bfloat16* m,
                                          int piece, int off) {
    uint32_t f[NB][4];
#pragma unroll
    for (int p = 0; p < NB; ++p) ldsm4t(f[p], smem_u32(m + p * piece + off));
    times_sum<NA, NB, 3>(d, first, a, f);
}
// (d0, d1) <- f (x0, x1) + (d0, d1)
__device__ __forceinline__ void fma_pair(float& d0, float& d1, float f, float x0, float x1) {
    const F2 v = fma2(f2s(f), f2(x0, x1), f2(d0, d1));
    d0 = f2lo(v), d1 = f2hi(v);
}
// s <- f s + d
__device__ __forceinline__ void fade_add(float (&s)[4], float f, const float (&d)[4]) {
    const F2 a = fma2(f2(s[0], s[1]), f2s(f), f2(d[0], d[1])), b = fma2(f2(s[2], s[3]), f2s(f), f2(d[2], d[3]));
    s[0] = f2lo(a), s[1] = f2hi(a), s[2] = f2lo(b), s[3] = f2hi(b);
}
// The walks over value columns.  ROPS: R is staged too; MATS: 16 x 16
// matrices (pieces) a chunk; SCS: factors a token.
template <typename IO, int N, bool ROPS, int MATS, int SCS>
struct Columns {
    static constexpr int KP = sizeof(IO) == 2 ? 1 : 3;           // pieces of K and R
    static constexpr int NW = N == 32 ? 2 : 4;                   // walking warps
    static constexpr int CW = 16 * NW, SLICES = N / CW, NST = 4;
    static constexpr int WALK = 32 * NW, THREADS = WALK + 32 * NST;
    static constexpr int BAR = WALK + 32;                        // threads of a stage's barriers
    static constexpr int LD = N + 8, PIECE = kChunk * LD;
    static constexpr int OPS = (ROPS ? 2 : 1) * KP * PIECE;
    static constexpr int LDV = KP == 1 ? CW + 8 : CW + 4, VEL = kChunk * LDV;   // V in the I/O type
    // bytes of a stage, in order
    static constexpr int S_OPS = OPS * 2, S_V = VEL * int(sizeof(IO)), S_MAT = MATS * kMat * 2;
    static constexpr int S_SC = (SCS + 1) * kChunk * 4;                         // factors, beta
    static constexpr int S_OWN = kChunk * 8 + 16 * 20 * 4;                      // the staging warp's
    static constexpr int STAGE = S_OPS + S_V + S_MAT + S_SC + S_OWN;
    static constexpr int SMEM = NST * STAGE;

    __nv_bfloat16* k;
    IO* v;
    __nv_bfloat16* mats;
    float *sc, *diag, *beta;
    float2* sums;
    __device__ __forceinline__ Columns(char* smem, int st) {
        char* p = smem + st * STAGE;
        k = reinterpret_cast<__nv_bfloat16*>(p);
        v = reinterpret_cast<IO*>(p + S_OPS);
        mats = reinterpret_cast<__nv_bfloat16*>(p + S_OPS + S_V);
        diag = reinterpret_cast<float*>(p + S_OPS + S_V + S_MAT);
        sums = reinterpret_cast<float2*>(diag + 16 * 20);
        beta = reinterpret_cast<float*>(sums + kChunk);
        sc = beta + kChunk;
    }
    __device__ __forceinline__ __nv_bfloat16* r() const { return k + KP * PIECE; }
    // a chunk's rows of every tensor (one warp)
    __device__ __forceinline__ void fetch(const IO* kp, const IO* rp, int64_t ks, const IO* vp, int64_t vs, int nt, bool vec,
                                          int lane) {
        copy_rows<IO, kChunk, CW>(v, Pitched<LDV>{}, vp, vs, nt, vec, lane);
        if constexpr (KP == 1) {
            copy_rows<IO, kChunk, N>(reinterpret_cast<IO*>(k), Pitched<LD>{}, kp, ks, nt, vec, lane);
            if constexpr (ROPS) copy_rows<IO, kChunk, N>(reinterpret_cast<IO*>(r()), Pitched<LD>{}, rp, ks, nt, vec, lane);
        }
        cp_async_commit();
        if constexpr (KP == 3) {
            split_rows<kChunk, N, 3>(k, Pitched<LD>{}, PIECE, reinterpret_cast<const float*>(kp), ks, nt, vec, lane);
            if constexpr (ROPS) split_rows<kChunk, N, 3>(r(), Pitched<LD>{}, PIECE, reinterpret_cast<const float*>(rp), ks, nt, vec, lane);
        }
        cp_async_wait();
        __syncwarp();
    }
};

// S^T of a warp from / to a state S[key][value]: tile n holds keys 8 n .. 8 n + 7
// of line lane / 4 (+ 8)
template <int N>
__device__ __forceinline__ void load_state(float (&S)[N / 8][4], const float* s, int lane) {
#pragma unroll
    for (int n = 0; n < N / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            S[n][i] = s != nullptr ? s[(8 * n + 2 * (lane % 4) + (i & 1)) * N + lane / 4 + (i >> 1) * 8] : 0.f;
}
template <int N>
__device__ __forceinline__ void store_state(float* s, const float (&S)[N / 8][4], int lane) {
#pragma unroll
    for (int n = 0; n < N / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[(8 * n + 2 * (lane % 4) + (i & 1)) * N + lane / 4 + (i >> 1) * 8] = S[n][i];
}
// The segments' kernel of the reverse mode: tcgen05.mma (wkv_delta_tc.cuh; 1735 us
// for 8 x 4096 tokens of 32 heads where mma.sync takes 1837), or mma.sync, as heads of
// other sizes and float32 take: heads of 128 and float32's pieces need more tiles
// than two CTAs an SM have room for, heads of 32 would leave half of each unused.
template <typename IO, int N>
constexpr bool kTcSegments = N == 64 && sizeof(IO) == 2;
// The states between segments as that kernel reads them: S[key][value], or
// S^T[value][key].  j: the warp's first value column.
template <typename IO, int N>
__device__ __forceinline__ void keep_state(float* s, int j, const float (&S)[N / 8][4], int lane) {
    if constexpr (kTcSegments<IO, N>) {
        store_state<N>(s + j, S, lane);
    } else {
#pragma unroll
        for (int n = 0; n < N / 8; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                *reinterpret_cast<float2*>(s + (j + lane / 4 + 8 * q) * N + 8 * n + 2 * (lane % 4)) =
                    make_float2(S[n][2 * q], S[n][2 * q + 1]);
    }
}

// The walk's state as a warp holds it, between the parts of a walk
template <int N>
__device__ __forceinline__ void hand_on(float* s, const float (&S)[N / 8][4], int lane) {
#pragma unroll
    for (int n = 0; n < N / 8; ++n)
        __stcg(reinterpret_cast<float4*>(s) + n * 32 + lane, make_float4(S[n][0], S[n][1], S[n][2], S[n][3]));
    __threadfence();
}
template <int N>
__device__ __forceinline__ void take_over(float (&S)[N / 8][4], const float* s, bool lost, int lane) {
#pragma unroll
    for (int n = 0; n < N / 8; ++n) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(s) + n * 32 + lane);
        S[n][0] = v.x, S[n][1] = v.y, S[n][2] = v.z, S[n][3] = v.w;
        if (lost) S[n][0] = S[n][1] = S[n][2] = S[n][3] = __int_as_float(0x7fffffff);
    }
}

// What a CTA works on: one walk (a head's slice of columns) over all tokens,
// or, where the walks would leave the last of several waves mostly empty, one
// part of a walk after another.  Tickets go through the first part of every
// walk, then the second: a part's predecessor was taken earlier, so somebody
// is at it or done with it, and by then it is nearly always done.  A wait ends
// after wait_ns; it leaves the error word, and NaN in that part and all that
// follow it.
constexpr uint32_t kLost = 0xffffffffu;   // of the parts that are done: one was given up
struct Task {
    int64_t walk, part;
    bool lost;   // the part before it never came
};
// The next task of the CTA (every thread calls; THREADS of them), false: none
// is left.  Publishes the one before: its state is written and fenced.
template <bool PARTS, int THREADS>
__device__ __forceinline__ bool next_task(const Args& a, int64_t walks, int64_t block, Task& t, bool first) {
    if constexpr (!PARTS) {
        t = Task{block, 0, false};
        return first;
    }
    __shared__ int64_t s_ticket;
    __shared__ int s_lost;
    bar_sync<THREADS>(kBarTask);
    if (threadIdx.x == 0) {
        if (!first)
            asm volatile("red.release.gpu.global.max.u32 [%0], %1;" ::"l"(a.done + t.walk), "r"(t.lost ? kLost : uint32_t(t.part + 1)) : "memory");
        const int64_t id = atomicAdd(a.ticket, 1u);
        s_ticket = id;
        s_lost = 0;
        if (id < walks * a.parts) {
            const uint32_t want = uint32_t(id / walks);
            uint64_t begin, now;
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(begin));
            uint32_t have = 0;
            while (true) {
                asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(have) : "l"(a.done + id % walks) : "memory");
                if (have >= want) break;
                asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
                if (now - begin > a.wait_ns) {
                    record_lost(a.control, uint32_t(id));
                    have = kLost;
                    break;
                }
            }
            s_lost = have == kLost;
        }
    }
    __syncwarp();
    bar_sync<THREADS>(kBarTask);
    t = Task{s_ticket % walks, s_ticket / walks, s_lost != 0};
    return t.part < a.parts;
}

// two neighbouring channels of a staged row, KP pieces `piece` elements apart
template <int KP>
__device__ __forceinline__ float2 staged_pair(const __nv_bfloat16* p, int piece) {
    float2 x = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = KP - 1; c >= 0; --c) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p + c * piece);
        x.x += __uint_as_float(w << 16), x.y += __uint_as_float(w & 0xffff0000u);
    }
    return x;
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
// Of each quad of lanes (two lines of a warp's tiles): does p hold in one of them?
__device__ __forceinline__ uint32_t quad_any(bool p) {
    uint32_t b = __ballot_sync(0xffffffffu, p);
    b |= b >> 1;
    return (b | b >> 2) & 0x11111111u;
}
// A walking warp's place: tokens [begin, end) of a head, columns from `column` on
template <typename G, int N, bool PARTS, bool BACK>
struct Reach {
    int64_t head, row, begin, end, values;   // row, values: of token 0, in per-head scalars and in values
    int column;
    __device__ __forceinline__ Reach(const Args& a, const Task& t, int warp) {
        head = t.walk / G::SLICES;
        const int64_t b = head / a.H, h = head % a.H;
        column = int(t.walk % G::SLICES) * G::CW + warp * 16;
        begin = PARTS ? (BACK ? a.parts - 1 - t.part : t.part) * a.part_len : 0;
        end = PARTS && begin + a.part_len < a.T ? begin + a.part_len : a.T;
        row = b * a.T * a.H + h;
        values = row * N + column;
    }
    // the state that the walk begins with: `given` (NULL: zeros), or what the part before left
    __device__ __forceinline__ void start(float (&S)[N / 8][4], const Args& a, const Task& t, const float* given, int lane) const {
        if (!PARTS || t.part == 0) load_state<N>(S, given == nullptr ? nullptr : given + head * N * N + column, lane);
        else take_over<N>(S, hand(a), t.lost, lane);
    }
    __device__ __forceinline__ float* hand(const Args& a) const { return a.hand + head * N * N + int64_t(column) * N; }
};
// Which of a warp's lines are not finite?  Of a quad of lanes, its two lines in
// neighbouring bits.  (0 times what is not finite is NaN.)
template <int N>
__device__ __forceinline__ uint32_t odd_lines(const float (&x)[N / 8][4]) {
    float z[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < N / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i >> 1] = fmaf(x[n][i], 0.f, z[i >> 1]);
    return quad_any(z[0] != 0.f) | quad_any(z[1] != 0.f) << 1;
}
// Was one of `lines` finite when the walk began?
template <int N, typename PLACE>
__device__ __noinline__ bool began_finite(const Args& a, const Task& t, const float* given, uint32_t lines) {
    float s[N / 8][4];
    PLACE(a, t, threadIdx.x / 32).start(s, a, t, given, threadIdx.x % 32);
    return (lines & ~odd_lines<N>(s)) != 0;
}

// steps of 16 in a chain of the tensor cores' additions.  float32 heads of 128
// with whole chains: y within 6.8e-7 of 64 bits, dw 2e-6; with chains of one
// 1.3e-7 and 5e-7.  bfloat16 keeps chains of 4 (heads of 64 whole; heads of 128
// dw 4e-7, was 8e-7, for 2% of the time).
template <typename IO>
constexpr int kChain = sizeof(IO) == 2 ? 4 : 1;

// CTAs an SM: two where the state's lines and the I/O type leave room (8 x 4096
// tokens of 32 heads of 64: two walks an SM share its issue slots, 429 us for
// 1.73 walks an SM where one walk alone takes 242)
template <typename IO, int N>
constexpr int kCtas = N <= 64 && sizeof(IO) == 2 ? 2 : 1;
// Two walks of heads of 64 in bfloat16 fit an SM with 128 registers a thread on
// average: the walking warps take 168 and the staging warps keep 88 (four
// warps each, 128 * 168 + 128 * 88 = 256 * 128, what the CTA has).
template <typename IO, int N>
constexpr bool kShareRegs = N == 64 && sizeof(IO) == 2;
template <typename IO, int N>
__device__ __forceinline__ void stager_regs() {
    if constexpr (kShareRegs<IO, N>) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
}
template <typename IO, int N>
__device__ __forceinline__ void walker_regs() {
    if constexpr (kShareRegs<IO, N>) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
}

// Outputs y (WANT_Y), or the errors e and the states between segments for the
// reverse mode (float32).
template <typename IO, int N, bool WANT_Y>
using ForwardShape = Columns<IO, N, WANT_Y, WANT_Y ? 6 : 3, 2>;

// A chunk's nt tokens of a warp's 16 columns one after another, from the staged rows:
// outputs y or errors e at `out` (the lane's first line).  w, beta: of its first token.
template <typename IO, int N, bool WANT_Y, typename OUT>
__device__ __forceinline__ void forward_tokens(const ForwardShape<IO, N, WANT_Y>& g, float (&S)[N / 8][4], int j0, int nt, const float* w,
                                               const float* beta, int64_t heads, OUT* out, int64_t vs, int lane) {
    using G = ForwardShape<IO, N, WANT_Y>;
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
        const __nv_bfloat16* kp = g.k + t * G::LD + 2 * (lane % 4);
        const IO* vp = g.v + t * G::LDV + j0 + lane / 4;
        const float a = expf(-w[t * heads]), be = beta[t * heads];
        float p[2] = {0.f, 0.f}, u[2];
#pragma unroll
        for (int n = 0; n < N / 8; ++n) {
            const float2 k = staged_pair<G::KP>(kp + 8 * n, G::PIECE);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                S[n][i] *= a;
                p[i >> 1] = fmaf(S[n][i], (i & 1) ? k.y : k.x, p[i >> 1]);
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            p[q] = to_f32(vp[8 * q]) - quad_sum(p[q]);
            u[q] = be * p[q];
        }
        float y[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < N / 8; ++n) {
            const float2 k = staged_pair<G::KP>(kp + 8 * n, G::PIECE);
            float2 r = make_float2(0.f, 0.f);
            if constexpr (WANT_Y) r = staged_pair<G::KP>(kp + (g.r() - g.k) + 8 * n, G::PIECE);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                S[n][i] = fmaf((i & 1) ? k.y : k.x, u[i >> 1], S[n][i]);
                if constexpr (WANT_Y) y[i >> 1] = fmaf(S[n][i], (i & 1) ? r.y : r.x, y[i >> 1]);
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if constexpr (WANT_Y) p[q] = quad_sum(y[q]);
            if (lane % 4 == 0) put(out + t * vs + 8 * q, p[q]);
        }
    }
}

// where the state behind the walk's last token goes
template <typename IO, int N, bool WANT_Y, bool PARTS, typename PLACE>
__device__ __forceinline__ void forward_end(const Args& a, const PLACE& p, const float (&S)[N / 8][4], int lane) {
    const int64_t nseg = (a.T + kSegment - 1) / kSegment;
    if (PARTS && p.end < a.T) {
        hand_on<N>(p.hand(a), S, lane);
    } else if constexpr (WANT_Y) {
        if (a.s_out != nullptr) store_state<N>(a.s_out + p.head * N * N + p.column, S, lane);
    } else {
        keep_state<IO, N>(a.s_seg + (p.head * (nseg + 1) + nseg) * N * N, p.column, S, lane);
    }
}
template <typename IO, int N, bool WANT_Y, bool PARTS>
__device__ __noinline__ void forward_again(const Args& a, char* smem, const Task& task) {
    using G = ForwardShape<IO, N, WANT_Y>;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t nseg = (a.T + kSegment - 1) / kSegment, vs = a.H * N;
    const Reach<G, N, PARTS, false> p(a, task, warp);
    float S[N / 8][4];
    p.start(S, a, task, a.s_in, lane);
    int st = 0;
#pragma unroll 1
    for (int64_t t0 = p.begin; t0 < p.end; t0 += kChunk, st = (st + 1) % G::NST) {
        const int nt = p.end - t0 < kChunk ? int(p.end - t0) : kChunk;
        const int64_t row = p.row + t0 * a.H, line = p.values + t0 * vs + lane / 4;
        if (!WANT_Y && t0 % kSegment == 0)
            keep_state<IO, N>(a.s_seg + (p.head * (nseg + 1) + t0 / kSegment) * N * N, p.column, S, lane);
        bar_sync<G::BAR>(kBarFull + st);
        if constexpr (WANT_Y)
            forward_tokens<IO, N, true>(G(smem, st), S, warp * 16, nt, a.w + row, a.beta + row, a.H, static_cast<IO*>(a.y) + line, vs, lane);
        else
            forward_tokens<IO, N, false>(G(smem, st), S, warp * 16, nt, a.w + row, a.beta + row, a.H, a.e + line, vs, lane);
        if (t0 + G::NST * kChunk < p.end) bar_arrive<G::BAR>(kBarFree + st);
    }
    forward_end<IO, N, WANT_Y, PARTS>(a, p, S, lane);
}

template <typename IO, int N, bool WANT_Y, bool PARTS>
__device__ __forceinline__ void forward_walk(const Args& a, char* smem, int64_t block) {
    using G = ForwardShape<IO, N, WANT_Y>;
    constexpr int KP = G::KP, LD = G::LD, C = kChain<IO>;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;

    const int64_t walks = a.B * a.H * G::SLICES, vs = a.H * N;
    Task task;
    bool first = true;

    if (warp >= G::NW) {
        stager_regs<IO, N>();
        const int st = warp - G::NW;
        const int64_t ks = a.Hk * N;
        G g(smem, st);
        for (; next_task<PARTS, G::THREADS>(a, walks, block, task, first); first = false) {
            const int64_t head = task.walk / G::SLICES, b = head / a.H, h = head % a.H, hk = h / (a.H / a.Hk);
            const int64_t begin = PARTS ? task.part * a.part_len : 0;
            const int64_t end = PARTS && begin + a.part_len < a.T ? begin + a.part_len : a.T;
            const IO* kp = static_cast<const IO*>(a.k) + (b * a.T * a.Hk + hk) * N;
            const IO* rp = static_cast<const IO*>(a.r) + (b * a.T * a.Hk + hk) * N;
            const IO* vp = static_cast<const IO*>(a.v) + (b * a.T * a.H + h) * N + task.walk % G::SLICES * G::CW;
            const float* wp = a.w + b * a.T * a.H + h;
            const float* bp = a.beta + b * a.T * a.H + h;
            bool again = false;
            do {
#pragma unroll 1
                for (int64_t t0 = begin + st * kChunk; t0 < end; t0 += G::NST * kChunk) {
                    const int nt = end - t0 < kChunk ? int(end - t0) : kChunk;
                    if (t0 >= begin + G::NST * kChunk) bar_sync<G::BAR>(kBarFree + st);
                    const float w = lane < nt ? wp[(t0 + lane) * a.H] : 0.f, be = lane < nt ? bp[(t0 + lane) * a.H] : 0.f;
                    g.fetch(kp + t0 * ks, rp + t0 * ks, ks, vp + t0 * vs, vs, nt, a.vec, lane);
                    // A, its inverse and P
                    const ChunkDecay d = chunk_decay<kChunk>(w, g.sums, lane);
                    if (lane < kChunk) {
                        g.beta[lane] = be;
                        g.sc[lane] = d.upto;
                        g.sc[kChunk + lane] = d.after * be;
                    }
                    __syncwarp();
                    float kk[2][4], rk[2][4];
                    gram<N, KP, KP, KP, kChain<IO>>(kk, g.k, g.k, G::PIECE, lane);
                    if constexpr (WANT_Y) gram<N, KP, KP, KP, kChain<IO>>(rk, g.r(), g.k, G::PIECE, lane);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float2 bs = pair_at(g.beta, n, lane);
                        const int s = 8 * n + 2 * (lane % 4);
                        const float2 s0 = g.sums[s], s1 = g.sums[s + 1];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int t = lane / 4 + 8 * q;
                            const float2 tt = g.sums[t];
                            const float g0 = decay_of(tt, s0) * bs.x, g1 = decay_of(tt, s1) * bs.y;
                            g.diag[t * 20 + s] = s < t ? g0 * kk[n][2 * q] : 0.f;
                            g.diag[t * 20 + s + 1] = s + 1 < t ? g1 * kk[n][2 * q + 1] : 0.f;
                            if constexpr (WANT_Y)
                                put_pieces<3>(g.mats + 3 * kMat, t, s, s <= t ? g0 * rk[n][2 * q] : 0.f,
                                              s + 1 <= t ? g1 * rk[n][2 * q + 1] : 0.f);
                        }
                    }
                    __syncwarp();
                    put_inverse(g.mats, g.diag, lane);
                    bar_arrive<G::BAR>(kBarFull + st);
                }
            } while (!again && (again = bar_or<G::THREADS>(kBarTask, false)));
        }
        return;
    }

    walker_regs<IO, N>();
    const int j0 = warp * 16;
    const int64_t nseg = (a.T + kSegment - 1) / kSegment;
    const int off_b = b_plain(lane, LD), off_t = b_trans(lane, LD), off_m = m_plain(lane);
    using Place = Reach<G, N, PARTS, false>;
    for (; next_task<PARTS, G::THREADS>(a, walks, block, task, first); first = false) {
        const Place here(a, task, warp);
        const int64_t end = here.end;
        float* keep = a.s_seg + here.head * (nseg + 1) * N * N;
        float S[N / 8][4];
        here.start(S, a, task, a.s_in, lane);
        int st = 0;
#pragma unroll 1
        for (int64_t t0 = here.begin; t0 < end; t0 += kChunk, st = (st + 1) % G::NST) {
            const int nt = end - t0 < kChunk ? int(end - t0) : kChunk;
            G g(smem, st);
            if (!WANT_Y && t0 % kSegment == 0) keep_state<IO, N>(keep + t0 / kSegment * N * N, here.column, S, lane);
            bar_sync<G::BAR>(kBarFull + st);
            // K S and R S, transposed
            float p[2][4], q[2][4], x[2][4];
            {
                Acc pa, qa;
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    uint32_t sp[3][4];
                    split_a<3>(S[2 * kk], S[2 * kk + 1], sp);
                    times<3, KP, 3, false>(pa, pa.template start<C>(p, kk), kk == 0, sp, g.k + kk * 16, G::PIECE, off_b);
                    if constexpr (WANT_Y)
                        times<3, KP, 3, false>(qa, qa.template start<C>(q, kk), kk == 0, sp, g.r() + kk * 16, G::PIECE, off_b);
                }
                pa.template finish<C>(p, N / 16);
                if constexpr (WANT_Y) qa.template finish<C>(q, N / 16);
            }
            load_lines(x, g.v + j0, G::LDV, lane);
            // X = V - g K S
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float2 gg = pair_at(g.sc, n, lane);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[n][i] = fmaf(-((i & 1) ? gg.y : gg.x), p[n][i], x[n][i]);
            }
            // E = (I + A)^-1 X
            float e[2][4];
            {
                uint32_t xp[3][4];
                split_a<3>(x[0], x[1], xp);
                Acc ea;
                times<3, 3, 3, false>(ea, true, true, xp, g.mats, kMat, off_m);
                ea.sum(e);
            }
            // S <- g_15 S + (G beta E)^T K
            {
                float u[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[n][i] = e[n][i];
                scale_tokens(u, g.sc + kChunk, lane);
                uint32_t up[3][4];
                split_a<3>(u[0], u[1], up);
                const float gl = g.sc[kChunk - 1];
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    float d[2][4];
                    times_add<3, KP>(d, true, up, g.k + kk * 16, G::PIECE, off_t);
                    fade_add(S[2 * kk], gl, d[0]);
                    fade_add(S[2 * kk + 1], gl, d[1]);
                }
            }
            const int64_t at = here.values + t0 * vs;
            if constexpr (!WANT_Y) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    store_half(a.e + at + 8 * n * vs, vs, nt - 8 * n, e[n], g.v, 0, false, lane);
            } else {
                // Y = g R S + P E
                uint32_t ep[3][4];
                split_a<3>(e[0], e[1], ep);
                Acc ya;
                times<3, 3, 3, false>(ya, true, true, ep, g.mats + 3 * kMat, kMat, off_m);
                float y[2][4];
                ya.sum(y);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float2 gg = pair_at(g.sc, n, lane);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[n][i] = fmaf((i & 1) ? gg.y : gg.x, q[n][i], y[n][i]);
                    // through the V tile's columns, which only this warp reads
                    store_half(static_cast<IO*>(a.y) + at + 8 * n * vs, vs, nt - 8 * n, y[n], g.v + 8 * n * G::LDV + j0, G::LDV, a.vec, lane);
                }
            }
            if (t0 + G::NST * kChunk < end) bar_arrive<G::BAR>(kBarFree + st);
        }
        const uint32_t odd = odd_lines<N>(S);
        if (bar_or<G::THREADS>(kBarTask, odd != 0 && began_finite<N, Place>(a, task, a.s_in, odd))) {
            forward_again<IO, N, WANT_Y, PARTS>(a, smem, task);
            continue;
        }
        forward_end<IO, N, WANT_Y, PARTS>(a, here, S, lane);
    }
}

template <typename IO, int N, bool WANT_Y, bool PARTS>
__global__ void __launch_bounds__(ForwardShape<IO, N, WANT_Y>::THREADS, kCtas<IO, N>) delta_forward_mma_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(16) char smem[];
    pdl_wait();
    forward_walk<IO, N, WANT_Y, PARTS>(a, smem, blockIdx.x);
}

}  // namespace delta
}  // namespace wkv
