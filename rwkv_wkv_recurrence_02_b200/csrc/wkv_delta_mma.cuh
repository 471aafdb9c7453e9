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
// A warp owns 16 value columns for the whole key axis and keeps S^T for them
// as mma accumulators (m = value, n = key).  The accumulator layout of one
// product is the A-operand layout of the next, so S^T -> K S -> E -> S^T
// never leaves the registers; K, R and V come from shared memory by ldmatrix.
// A, its inverse and P do not depend on the state: for each block of 64 or 32
// tokens the CTA's warps form those of one chunk each, then every warp walks
// the block's chunks.
//
// Accuracy: a float32 operand is the sum of three bfloat16 pieces (24 bits);
// products of pieces up to 2^-16 of the leading one are taken, each order in
// its own accumulator.  bfloat16 inputs are one piece, exact: three products
// for what reaches the state.  What only reaches a bfloat16 output takes the
// orders up to 2^-8 (an error of 2^-17 against the output's own 2^-9).  The state is
// updated by a float32 multiply-add of the chunk's sum, so the accumulators'
// truncation does not add up along T.
#pragma once

#include "wkv_delta.cuh"

namespace wkv {
namespace delta {

constexpr int kChunk = 16;     // tokens of a chunk: one k step of an mma
constexpr int kMatLd = 24;     // row pitch of the 16 x 16 matrices (48 bytes: ldmatrix rows in distinct banks)

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
__device__ __forceinline__ void stsm4t(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
                 :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
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
constexpr int kBarFull = 1, kBarFree = 3, kBarStage = 5;   // full and free: one for each of two stages

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

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

// Rows t0 .. of W elements to shared rows of LD elements: 16-byte
// asynchronous copies, or element copies where the addresses do not allow
// them; rows from nt on are zero.
template <typename IO, int BLK, int W, int LD, int THREADS>
__device__ __forceinline__ void copy_rows(IO* dst, const IO* src, int64_t stride, int nt, bool vec, int tid) {
    if (vec) {
        constexpr int PER = 16 / int(sizeof(IO)), ROWV = W / PER;
#pragma unroll
        for (int i = tid; i < BLK * ROWV; i += THREADS) {
            const int t = i / ROWV, c = (i % ROWV) * PER;
            cp_async16(smem_u32(dst + t * LD + c), src + (t < nt ? t : 0) * stride + c, t < nt);
        }
    } else {
        for (int i = tid; i < BLK * W; i += THREADS) {
            const int t = i / W, c = i % W;
            IO x;
            if constexpr (sizeof(IO) == 4) x = 0.f;
            else x = __ushort_as_bfloat16(0);
            if (t < nt) x = src[t * stride + c];
            dst[t * LD + c] = x;
        }
    }
}

// float32 rows as NP arrays of bfloat16 pieces, `piece` elements apart
template <int BLK, int W, int LDS, int LDD, int NP, int THREADS>
__device__ __forceinline__ void split_rows(__nv_bfloat16* dst, int piece, const float* src, int tid) {
#pragma unroll 4
    for (int i = tid; i < BLK * W / 2; i += THREADS) {
        const int t = i / (W / 2), c = (i % (W / 2)) * 2;
        const float2 x = *reinterpret_cast<const float2*>(src + t * LDS + c);
        uint32_t p[NP];
        split2<NP>(x.x, x.y, p);
#pragma unroll
        for (int q = 0; q < NP; ++q) *reinterpret_cast<uint32_t*>(dst + q * piece + t * LDD + c) = p[q];
    }
}

// (16 tokens x N) (N x 16 tokens)^T of two staged arrays of KX and KY pieces,
// the products of the first ORD orders: C[t][s] = x_t . y_s
template <int N, int KX, int KY, int ORD>
__device__ __forceinline__ void gram(float (&c)[2][4], const __nv_bfloat16* x, const __nv_bfloat16* y, int piece, int lane) {
    constexpr int LD = N + 8;
    // A: rows t, keys; B: rows s, keys
    bool first = true;
    const int ra = (lane & 7) + ((lane >> 3) & 1) * 8, ca = (lane >> 4) * 8;
    const int rb = (lane & 7) + (lane >> 4) * 8, cb = ((lane >> 3) & 1) * 8;
#pragma unroll
    for (int kk = 0; kk < N / 16; ++kk) {
        uint32_t a[KX][4], b[KY][4];
#pragma unroll
        for (int p = 0; p < KX; ++p) ldsm4(a[p], smem_u32(x + p * piece + ra * LD + kk * 16 + ca));
#pragma unroll
        for (int p = 0; p < KY; ++p) ldsm4(b[p], smem_u32(y + p * piece + rb * LD + kk * 16 + cb));
#pragma unroll
        for (int o = ORD - 1; o >= 0; --o)
#pragma unroll
            for (int p = 0; p < KX && p <= o; ++p)
                if (o - p < KY) {
                    mma2(c, a[p], b[o - p], first);
                    first = false;
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

// Decays of a chunk (one warp; lane % 16 is a token): gam[t][s] = product of
// the decays of tokens s + 1 .. t (0 above the diagonal; row pitch 17), the
// products up to a token and after it.
struct ChunkDecay {
    float upto, after;
};
__device__ __forceinline__ ChunkDecay chunk_decay(const float* w, float* gam, int lane) {
    const int tl = lane % 16;
    const float al = expf(-w[tl]);
    ChunkDecay d{0.f, 0.f};
    float run = 1.f;
#pragma unroll
    for (int t = 0; t < kChunk; ++t) {
        const float at = __shfl_sync(0xffffffffu, al, t);
        d.after = t == tl ? 1.f : d.after * at;
        run *= at;
        if (t == tl) d.upto = run;
        if (lane < 16) gam[t * 17 + tl] = d.after;
    }
    return d;
}

// (v0, v1) of row t, columns s, s + 1 into the pieces of a 16 x 16 matrix
template <int NP>
__device__ __forceinline__ void put_pieces(__nv_bfloat16* m, int t, int s, float v0, float v1) {
    uint32_t p[NP];
    split2<NP>(v0, v1, p);
#pragma unroll
    for (int q = 0; q < NP; ++q) *reinterpret_cast<uint32_t*>(m + q * kChunk * kMatLd + t * kMatLd + s) = p[q];
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
        for (int q = 0; q < 3; ++q)
            m[q * kChunk * kMatLd + t * kMatLd + lane % 16] = __ushort_as_bfloat16(static_cast<unsigned short>(p[q]));
    }
}

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

// Such a tile to rows of global memory (row t at out + t * stride), rows
// below nt.  bfloat16 goes through `rows`, a staged tile that only this warp
// uses, to 16-byte stores.
template <typename OUT, typename IO>
__device__ __forceinline__ void store_lines(OUT* out, int64_t stride, int nt, const float (&x)[2][4], IO* rows, int ld,
                                            bool vec, int lane) {
    if constexpr (sizeof(OUT) == 2) {
        uint32_t f[4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                const __nv_bfloat162 v2 = __floats2bfloat162_rn(x[n][2 * hrow], x[n][2 * hrow + 1]);
                f[2 * n + hrow] = *reinterpret_cast<const uint32_t*>(&v2);
            }
        const int m = lane >> 3;
        stsm4t(smem_u32(rows + ((lane & 7) + (m >> 1) * 8) * ld + (m & 1) * 8), f);
        __syncwarp();
        const int t = lane / 2, col = (lane % 2) * 8;
        const uint4 v4 = *reinterpret_cast<const uint4*>(rows + t * ld + col);
        if (t < nt) {
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
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 8 * n + 2 * (lane % 4) + (i & 1);
                if (t < nt) out[t * stride + lane / 4 + (i >> 1) * 8] = x[n][i];
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
// (2^-8 of it, so what their additions round off is 2^-8 of a float32 step).
struct Acc {
    float hi[2][4], lo[2][4];
    __device__ __forceinline__ void sum(float (&x)[2][4], bool has_lo = true) const {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[n][i] = has_lo ? hi[n][i] + lo[n][i] : hi[n][i];
    }
};
// acc (+)= A (16 x 16) B (16 x 16) of NA and NB pieces, orders below ORD.  B's
// pieces lie `piece` elements apart; off: this lane's offset (b_plain, b_trans).
template <int NA, int NB, int ORD, bool TRANS>
__device__ __forceinline__ void times(Acc& acc, bool first, const uint32_t (&a)[NA][4], const __nv_bfloat16* m, int piece,
                                      int off) {
    bool lo_first = first;
#pragma unroll
    for (int p = 0; p < NB && p < ORD; ++p) {
        uint32_t f[4];
        if constexpr (TRANS) ldsm4t(f, smem_u32(m + p * piece + off));
        else ldsm4(f, smem_u32(m + p * piece + off));
#pragma unroll
        for (int i = 0; i < NA && i + p < ORD; ++i) {
            if (i + p == 0) {
                mma2(acc.hi, a[i], f, first);
            } else {
                mma2(acc.lo, a[i], f, lo_first);
                lo_first = false;
            }
        }
    }
}
// d (+)= A B into one accumulator, smallest orders first
template <int NA, int NB>
__device__ __forceinline__ void times_add(float (&d)[2][4], bool first, const uint32_t (&a)[NA][4], const __nv_bfloat16* m,
                                          int piece, int off) {
    uint32_t f[NB][4];
#pragma unroll
    for (int p = 0; p < NB; ++p) ldsm4t(f[p], smem_u32(m + p * piece + off));
#pragma unroll
    for (int o = 2; o >= 0; --o)
#pragma unroll
        for (int p = 0; p < NB && p <= o; ++p)
            if (o - p < NA) {
                mma2(d, a[o - p], f[p], first);
                first = false;
            }
}
// s <- f s + d
__device__ __forceinline__ void fade_add(float (&s)[4], float f, const float (&d)[4]) {
    const F2 a = fma2(f2(s[0], s[1]), f2s(f), f2(d[0], d[1])), b = fma2(f2(s[2], s[3]), f2s(f), f2(d[2], d[3]));
    s[0] = f2lo(a), s[1] = f2hi(a), s[2] = f2lo(b), s[3] = f2hi(b);
}
// shared-memory offsets (elements) of this lane in a B operand: rows as they
// lie (row = column of the product) and transposed (row = its k)
__device__ __forceinline__ int b_plain(int lane, int ld) { return ((lane & 7) + (lane >> 4) * 8) * ld + ((lane >> 3) & 1) * 8; }
__device__ __forceinline__ int b_trans(int lane, int ld) { return ((lane & 7) + ((lane >> 3) & 1) * 8) * ld + (lane >> 4) * 8; }

// sum over this warp's 16 lines of x * y for each token of the chunk, to
// out[token * stride] (tokens below nt)
__device__ __forceinline__ void token_sums(float* out, int64_t stride, int nt, const float (&x)[2][4], const float (&y)[2][4],
                                           int lane) {
    float s[2][2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int q = 0; q < 2; ++q) s[n][q] = fmaf(x[n][q], y[n][q], x[n][q + 2] * y[n][q + 2]);
    // lanes 4 apart hold the same tokens: halve what a lane carries, then the lanes
    const bool b0 = lane & 4, b1 = lane & 8;
    float u[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) u[q] = (b0 ? s[1][q] : s[0][q]) + __shfl_xor_sync(0xffffffffu, b0 ? s[0][q] : s[1][q], 4);
    float v = (b1 ? u[1] : u[0]) + __shfl_xor_sync(0xffffffffu, b1 ? u[0] : u[1], 8);
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    const int t = (b0 ? 8 : 0) + 2 * (lane % 4) + (b1 ? 1 : 0);
    if (lane < 16 && t < nt) out[t * stride] = v;
}

// Shared memory of the two walks over value columns: K and R with V (or dY),
// two stages, each with its chunks' matrices.  ROPS: R is staged too; MATS:
// 16 x 16 matrices (pieces) a chunk; SCS: factors a token; VT: tiles of values
// (V or dY, V).
template <typename IO, int N, int NW, bool ROPS, int MATS, int SCS, int VT = 1>
struct MmaColumns {
    static constexpr int KP = sizeof(IO) == 2 ? 1 : 3;           // pieces of K and R
    static constexpr int CW = 16 * NW, SLICES = N / CW;
    static constexpr int WALK = 32 * NW, STAGERS = 64, THREADS = WALK + STAGERS;
    // tokens staged at a time: two CTAs of 64 channels fit an SM
    static constexpr int BLK = KP == 3 || N == 128 ? 32 : 64;
    static constexpr int NCH = BLK / kChunk;
    static constexpr int LD = N + 8, PIECE = BLK * LD;
    static constexpr int OPS = (ROPS ? 2 : 1) * KP * PIECE;
    static constexpr int LDV = KP == 1 ? CW + 8 : CW + 4, VEL = BLK * LDV;   // V in the I/O type
    static constexpr int LDR = N, ROW = BLK * LDR;                           // raw float32 rows
    static constexpr int MAT = kChunk * kMatLd;
    // bytes of a stage, in order
    static constexpr int S_OPS = OPS * 2, S_V = VT * VEL * int(sizeof(IO)), S_MAT = NCH * MATS * MAT * 2;
    static constexpr int S_SC = (2 + SCS) * BLK * 4;                         // w, beta, factors
    static constexpr int STAGE = S_OPS + S_V + S_MAT + S_SC;
    static constexpr int B_RAW = KP == 1 ? 0 : (ROPS ? 2 : 1) * ROW * 4;
    static constexpr int SCR = 16 * 17 + 8 + 16 * 20;                        // floats of a staging warp
    static constexpr int SMEM = 2 * STAGE + B_RAW + STAGERS / 32 * SCR * 4;

    __nv_bfloat16* k;
    IO* v;
    __nv_bfloat16* mats;
    float *w, *beta, *sc;
    __device__ __forceinline__ MmaColumns(char* smem, int st) {
        char* p = smem + st * STAGE;
        k = reinterpret_cast<__nv_bfloat16*>(p);
        v = reinterpret_cast<IO*>(p + S_OPS);
        mats = reinterpret_cast<__nv_bfloat16*>(p + S_OPS + S_V);
        w = reinterpret_cast<float*>(p + S_OPS + S_V + S_MAT);
        beta = w + BLK;
        sc = w + 2 * BLK;
    }
    __device__ __forceinline__ __nv_bfloat16* r() const { return k + KP * PIECE; }
    __device__ __forceinline__ float* scratch(char* smem, int i) const {
        return reinterpret_cast<float*>(smem + 2 * STAGE + B_RAW) + i * SCR;
    }
    // rows t0 .. of every tensor (the staging warps)
    __device__ __forceinline__ void fetch(char* smem, const IO* kp, const IO* rp, int64_t ks, const IO* vp, const IO* vp2,
                                          int64_t vs, const float* wp, const float* bp, int64_t H, int64_t t0, int nt, bool vec, int tid) {
        if constexpr (KP == 1) {
            copy_rows<IO, BLK, N, LD, STAGERS>(reinterpret_cast<IO*>(k), kp + t0 * ks, ks, nt, vec, tid);
            if constexpr (ROPS) copy_rows<IO, BLK, N, LD, STAGERS>(reinterpret_cast<IO*>(r()), rp + t0 * ks, ks, nt, vec, tid);
        } else {
            float* raw = reinterpret_cast<float*>(smem + 2 * STAGE);
            copy_rows<float, BLK, N, LDR, STAGERS>(raw, reinterpret_cast<const float*>(kp) + t0 * ks, ks, nt, vec, tid);
            if constexpr (ROPS)
                copy_rows<float, BLK, N, LDR, STAGERS>(raw + ROW, reinterpret_cast<const float*>(rp) + t0 * ks, ks, nt, vec, tid);
        }
        copy_rows<IO, BLK, CW, LDV, STAGERS>(v, vp + t0 * vs, vs, nt, vec, tid);
        if constexpr (VT == 2) copy_rows<IO, BLK, CW, LDV, STAGERS>(v + VEL, vp2 + t0 * vs, vs, nt, vec, tid);
        for (int t = tid; t < BLK; t += STAGERS) {
            w[t] = t < nt ? wp[(t0 + t) * H] : 0.f;
            beta[t] = t < nt ? bp[(t0 + t) * H] : 0.f;
        }
        cp_async_commit();
        cp_async_wait();
        bar_sync<STAGERS>(kBarStage);
        if constexpr (KP == 3) {
            const float* raw = reinterpret_cast<const float*>(smem + 2 * STAGE);
            split_rows<BLK, N, LDR, LD, 3, STAGERS>(k, PIECE, raw, tid);
            if constexpr (ROPS) split_rows<BLK, N, LDR, LD, 3, STAGERS>(r(), PIECE, raw + ROW, tid);
            bar_sync<STAGERS>(kBarStage);
        }
    }
};

// what only reaches y takes this many orders
template <typename IO>
constexpr int kOutOrders = sizeof(IO) == 2 ? 2 : 3;

// Outputs y (WANT_Y) or the errors e for the reverse mode (float32).  Two
// warps stage and prepare a block ahead; the others walk.
template <typename IO, int N, int NW, bool WANT_Y>
using ForwardShape = MmaColumns<IO, N, NW, WANT_Y, 3 + (WANT_Y ? kOutOrders<IO> : 0), 2>;

template <typename IO, int N, int NW, bool WANT_Y>
__global__ void __launch_bounds__(ForwardShape<IO, N, NW, WANT_Y>::THREADS, N == 64 && sizeof(IO) == 2 ? 2 : 1)
delta_forward_mma_kernel(const Args a) {
    using G = ForwardShape<IO, N, NW, WANT_Y>;
    constexpr int KP = G::KP, PP = kOutOrders<IO>, LD = G::LD, NT = N / 8, BLK = G::BLK, MATS = 3 + (WANT_Y ? PP : 0);
    extern __shared__ __align__(16) char smem[];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;

    const int64_t head = blockIdx.x / G::SLICES;
    const int slice = int(blockIdx.x % G::SLICES) * G::CW;
    const int64_t b = head / a.H, h = head % a.H, hk = h / (a.H / a.Hk);
    const int64_t vs = a.H * N;
    const int64_t vbase = (b * a.T * a.H + h) * N + slice;

    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp >= NW) {
        const int64_t ks = a.Hk * N;
        const IO* kp = static_cast<const IO*>(a.k) + (b * a.T * a.Hk + hk) * N;
        const IO* rp = static_cast<const IO*>(a.r) + (b * a.T * a.Hk + hk) * N;
        const int tl = lane % 16;
        int st = 0;
        for (int64_t t0 = 0; t0 < a.T; t0 += BLK, st ^= 1) {
            const int nt = a.T - t0 < BLK ? int(a.T - t0) : BLK;
            G g(smem, st);
            if (t0 >= 2 * BLK) bar_sync<G::THREADS>(kBarFree + st);
            g.fetch(smem, kp, rp, ks, static_cast<const IO*>(a.v) + vbase, nullptr, vs, a.w + b * a.T * a.H + h,
                    a.beta + b * a.T * a.H + h, a.H, t0, nt, a.vec, tid - G::WALK);
            float* gam = g.scratch(smem, warp - NW);
            float* amat = gam + 16 * 17 + 8;
            // A, its inverse and P
            for (int c = warp - NW; c * kChunk < nt; c += G::STAGERS / 32) {
                const ChunkDecay d = chunk_decay(g.w + c * kChunk, gam, lane);
                if (lane < 16) {
                    g.sc[c * kChunk + tl] = d.upto;
                    g.sc[BLK + c * kChunk + tl] = d.after * g.beta[c * kChunk + tl];
                }
                __syncwarp();
                const __nv_bfloat16* kc = g.k + c * kChunk * LD;
                float kk[2][4], rk[2][4];
                gram<N, KP, KP, KP>(kk, kc, kc, G::PIECE, lane);
                if constexpr (WANT_Y) gram<N, KP, KP, KP>(rk, g.r() + c * kChunk * LD, kc, G::PIECE, lane);
                __nv_bfloat16* tm = g.mats + c * MATS * G::MAT;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float2 bs = pair_at(g.beta + c * kChunk, n, lane);
                    const int s = 8 * n + 2 * (lane % 4);
#pragma unroll
                    for (int hrow = 0; hrow < 2; ++hrow) {
                        const int t = lane / 4 + 8 * hrow;
                        const float g0 = gam[t * 17 + s] * bs.x, g1 = gam[t * 17 + s + 1] * bs.y;
                        amat[t * 20 + s] = s < t ? g0 * kk[n][2 * hrow] : 0.f;
                        amat[t * 20 + s + 1] = s + 1 < t ? g1 * kk[n][2 * hrow + 1] : 0.f;
                        if constexpr (WANT_Y)
                            put_pieces<PP>(tm + 3 * G::MAT, t, s, g0 * rk[n][2 * hrow], g1 * rk[n][2 * hrow + 1]);
                    }
                }
                __syncwarp();
                put_inverse(tm, amat, lane);
                __syncwarp();
            }
            bar_arrive<G::THREADS>(kBarFull + st);
        }
        return;
    }

    const int j0 = warp * 16;
    // S^T: tile n holds keys 8 n .. 8 n + 7 of values j0 + lane / 4 (+ 8)
    float S[NT][4];
    {
        const float* s = a.s_in + head * N * N + slice + j0 + lane / 4;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = 8 * n + 2 * (lane % 4) + (i & 1);
                S[n][i] = a.s_in != nullptr ? s[key * N + (i >> 1) * 8] : 0.f;
            }
    }
    const int off_b = b_plain(lane, LD), off_t = b_trans(lane, LD), off_m = b_plain(lane, kMatLd);
    int st = 0;
    for (int64_t t0 = 0; t0 < a.T; t0 += BLK, st ^= 1) {
        const int nt = a.T - t0 < BLK ? int(a.T - t0) : BLK;
        G g(smem, st);
        bar_sync<G::THREADS>(kBarFull + st);
#pragma unroll 1
        for (int c = 0; c * kChunk < nt; ++c) {
            const __nv_bfloat16* kc = g.k + c * kChunk * LD;
            const __nv_bfloat16* rc = g.r() + c * kChunk * LD;
            const __nv_bfloat16* tm = g.mats + c * MATS * G::MAT;
            const float* gt = g.sc + c * kChunk;
            // K S and R S, transposed
            Acc pa, qa;
#pragma unroll
            for (int kk = 0; kk < N / 16; ++kk) {
                uint32_t sp[3][4];
                split_a<3>(S[2 * kk], S[2 * kk + 1], sp);
                times<3, KP, 3, false>(pa, kk == 0, sp, kc + kk * 16, G::PIECE, off_b);
                if constexpr (WANT_Y) times<3, KP, PP, false>(qa, kk == 0, sp, rc + kk * 16, G::PIECE, off_b);
            }
            // X = V - g K S
            float x[2][4], p[2][4];
            float2 gg[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) gg[n] = pair_at(gt, n, lane);
            load_lines(x, g.v + c * kChunk * G::LDV + j0, G::LDV, lane);
            pa.sum(p);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[n][i] = fmaf(-((i & 1) ? gg[n].y : gg[n].x), p[n][i], x[n][i]);
            // E = (I + A)^-1 X
            float e[2][4];
            {
                uint32_t xp[3][4];
                split_a<3>(x[0], x[1], xp);
                Acc ea;
                times<3, 3, 3, false>(ea, true, xp, tm, G::MAT, off_m);
                ea.sum(e);
            }
            // S <- g_15 S + (G beta E)^T K
            {
                float u[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[n][i] = e[n][i];
                scale_tokens(u, gt + BLK, lane);
                uint32_t up[3][4];
                split_a<3>(u[0], u[1], up);
                const float gl = gt[kChunk - 1];
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    float d[2][4];
                    times_add<3, KP>(d, true, up, kc + kk * 16, G::PIECE, off_t);
                    fade_add(S[2 * kk], gl, d[0]);
                    fade_add(S[2 * kk + 1], gl, d[1]);
                }
            }
            const int64_t at = vbase + (t0 + c * kChunk) * vs + j0;
            if constexpr (!WANT_Y) {
                store_lines(a.e + at, vs, nt - c * kChunk, e, g.v, 0, false, lane);
            } else {
                // Y = g R S + P E
                uint32_t ep[PP][4];
                split_a<PP>(e[0], e[1], ep);
                Acc ya;
                times<PP, PP, PP, false>(ya, true, ep, tm + 3 * G::MAT, G::MAT, off_m);
                float y[2][4], q[2][4];
                qa.sum(q);
                ya.sum(y);
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[n][i] = fmaf((i & 1) ? gg[n].y : gg[n].x, q[n][i], y[n][i]);
                // through the V tile's columns, which only this warp reads
                store_lines(static_cast<IO*>(a.y) + at, vs, nt - c * kChunk, y, g.v + c * kChunk * G::LDV + j0, G::LDV, a.vec,
                            lane);
            }
        }
        if (t0 + 2 * BLK < a.T) bar_arrive<G::THREADS>(kBarFree + st);
    }
    if (WANT_Y && a.s_out != nullptr) {
        float* s = a.s_out + head * N * N + slice + j0 + lane / 4;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[(8 * n + 2 * (lane % 4) + (i & 1)) * N + (i >> 1) * 8] = S[n][i];
    }
}

}  // namespace delta
}  // namespace wkv
