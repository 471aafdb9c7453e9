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
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// (x, y) as NP packed bfloat16 pairs whose sum is the pair to 8 NP bits
template <int NP>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&p)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        p[i] = *reinterpret_cast<const uint32_t*>(&h);
        if (i + 1 < NP) {
            x -= __uint_as_float(p[i] << 16);
            y -= __uint_as_float(p[i] & 0xffff0000u);
        }
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

// float32 rows as three arrays of bfloat16 pieces, PIECE elements apart
template <int BLK, int W, int LDS, int LDD, int THREADS>
__device__ __forceinline__ void split_rows(__nv_bfloat16* dst, int piece, const float* src, int tid) {
#pragma unroll 4
    for (int i = tid; i < BLK * W / 2; i += THREADS) {
        const int t = i / (W / 2), c = (i % (W / 2)) * 2;
        const float2 x = *reinterpret_cast<const float2*>(src + t * LDS + c);
        uint32_t p[3];
        split2<3>(x.x, x.y, p);
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<uint32_t*>(dst + q * piece + t * LDD + c) = p[q];
    }
}

// (16 tokens x N) (N x 16 tokens)^T of two staged arrays of KX and KY pieces,
// the products of the first ORD orders: C[t][s] = x_t . y_s
template <int N, int KX, int KY, int ORD>
__device__ __forceinline__ void gram(float (&c)[2][4], const __nv_bfloat16* x, const __nv_bfloat16* y, int piece, int lane) {
    constexpr int LD = N + 8;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[n][i] = 0.f;
    // A: rows t, keys; B: rows s, keys
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
                    mma(c[0], a[p], b[o - p][0], b[o - p][1]);
                    mma(c[1], a[p], b[o - p][2], b[o - p][3]);
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

template <int NP>
__device__ __forceinline__ void sum_orders(float (&x)[2][4], const float (&o)[NP][2][4]) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float s = o[NP - 1][n][i];
#pragma unroll
            for (int p = NP - 2; p >= 0; --p) s += o[p][n][i];
            x[n][i] = s;
        }
}

template <typename IO, int N, int NW, bool WANT_Y>
struct MmaForward {
    static constexpr int KP = sizeof(IO) == 2 ? 1 : 3;           // pieces of K and R
    static constexpr int PP = sizeof(IO) == 2 ? 2 : 3;           // orders of what only reaches y
    static constexpr int CW = 16 * NW, SLICES = N / CW, THREADS = 32 * NW;
    // tokens staged at a time: as many as fit
    static constexpr int BLK = KP == 3 && N == 128 ? 32 : 64;
    static constexpr int LD = N + 8;
    static constexpr int PIECE = BLK * LD;
    static constexpr int OPS = (WANT_Y ? 2 : 1) * KP * PIECE;    // K (and R), bfloat16
    static constexpr int LDV = KP == 1 ? CW + 8 : CW + 4;
    static constexpr int VEL = BLK * LDV;                     // V, in the I/O type
    static constexpr int LDR = N;                                // raw float32 rows
    static constexpr int MAT = kChunk * kMatLd;
    static constexpr int NCH = BLK / kChunk;
    // bytes
    static constexpr int B_OPS = OPS * 2 * (KP == 1 ? 2 : 1);
    static constexpr int B_RAW = KP == 1 ? 0 : (WANT_Y ? 2 : 1) * BLK * LDR * 4;
    static constexpr int B_V = 2 * VEL * int(sizeof(IO));
    static constexpr int B_MAT = NCH * (3 + (WANT_Y ? PP : 0)) * MAT * 2;
    static constexpr int B_SC = 2 * 2 * BLK * 4 + 2 * BLK * 4;
    static constexpr int B_SCR = NW * (16 * 17 + 16 * 20 + 12) * 4;
    static constexpr int SMEM = B_OPS + B_RAW + B_V + B_MAT + B_SC + B_SCR;
};

// Outputs y (WANT_Y) or the errors e for the reverse mode (float32).
template <typename IO, int N, int NW, bool WANT_Y>
__global__ void __launch_bounds__(32 * NW) delta_forward_mma_kernel(const Args a) {
    using G = MmaForward<IO, N, NW, WANT_Y>;
    constexpr int KP = G::KP, PP = G::PP, LD = G::LD, NT = N / 8, BLK = G::BLK;
    extern __shared__ __align__(16) char smem_raw[];
    __nv_bfloat16* ops = reinterpret_cast<__nv_bfloat16*>(smem_raw);
    float* raw = reinterpret_cast<float*>(smem_raw + G::B_OPS);
    IO* vbuf = reinterpret_cast<IO*>(smem_raw + G::B_OPS + G::B_RAW);
    __nv_bfloat16* mats = reinterpret_cast<__nv_bfloat16*>(smem_raw + G::B_OPS + G::B_RAW + G::B_V);
    float* wb = reinterpret_cast<float*>(smem_raw + G::B_OPS + G::B_RAW + G::B_V + G::B_MAT);   // [2][w, beta][64]
    float* sc = wb + 4 * BLK;                                                                 // [g, G beta][64]
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    float* gam = sc + 2 * BLK + warp * (16 * 17 + 16 * 20 + 12);
    float* amat = gam + 16 * 17 + 8;   // 16-byte aligned: 280 floats on

    const int64_t head = blockIdx.x / G::SLICES;
    const int slice = int(blockIdx.x % G::SLICES) * G::CW;
    const int64_t b = head / a.H, h = head % a.H, hk = h / (a.H / a.Hk);
    const int64_t ks = a.Hk * N, vs = a.H * N;
    const IO* kp = static_cast<const IO*>(a.k) + (b * a.T * a.Hk + hk) * N;
    const IO* rp = static_cast<const IO*>(a.r) + (b * a.T * a.Hk + hk) * N;
    const int64_t vbase = (b * a.T * a.H + h) * N + slice;
    const IO* vp = static_cast<const IO*>(a.v) + vbase;
    const float* wp = a.w + b * a.T * a.H + h;
    const float* bp = a.beta + b * a.T * a.H + h;
    const int j0 = warp * 16;

    asm volatile("griddepcontrol.wait;" ::: "memory");

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

    auto fetch = [&](int64_t t0, int st) {
        const int nt = a.T - t0 < BLK ? int(a.T - t0) : BLK;
        if constexpr (KP == 1) {
            copy_rows<IO, BLK, N, LD, G::THREADS>(reinterpret_cast<IO*>(ops + st * G::OPS), kp + t0 * ks, ks, nt, a.vec, tid);
            if constexpr (WANT_Y)
                copy_rows<IO, BLK, N, LD, G::THREADS>(reinterpret_cast<IO*>(ops + st * G::OPS + G::PIECE), rp + t0 * ks, ks, nt,
                                                 a.vec, tid);
        } else {
            copy_rows<float, BLK, N, G::LDR, G::THREADS>(raw, reinterpret_cast<const float*>(kp) + t0 * ks, ks, nt, a.vec, tid);
            if constexpr (WANT_Y)
                copy_rows<float, BLK, N, G::LDR, G::THREADS>(raw + BLK * G::LDR, reinterpret_cast<const float*>(rp) + t0 * ks,
                                                        ks, nt, a.vec, tid);
        }
        copy_rows<IO, BLK, G::CW, G::LDV, G::THREADS>(vbuf + st * G::VEL, vp + t0 * vs, vs, nt, a.vec, tid);
        for (int t = tid; t < BLK; t += G::THREADS) {
            wb[st * 2 * BLK + t] = t < nt ? wp[(t0 + t) * a.H] : 0.f;
            wb[(st * 2 + 1) * BLK + t] = t < nt ? bp[(t0 + t) * a.H] : 0.f;
        }
        cp_async_commit();
    };

    // A, its inverse and P of one chunk (one warp)
    auto prepare = [&](int c, const __nv_bfloat16* kb, const __nv_bfloat16* rb, const float* ws) {
        const int tl = lane % 16;
        const ChunkDecay d = chunk_decay(ws + c * kChunk, gam, lane);
        if (lane < 16) {
            sc[c * kChunk + tl] = d.upto;
            sc[BLK + c * kChunk + tl] = d.after * ws[BLK + c * kChunk + tl];
        }
        __syncwarp();
        float kk[2][4], rk[2][4];
        gram<N, KP, KP, KP>(kk, kb + c * kChunk * LD, kb + c * kChunk * LD, G::PIECE, lane);
        if constexpr (WANT_Y) gram<N, KP, KP, KP>(rk, rb + c * kChunk * LD, kb + c * kChunk * LD, G::PIECE, lane);
        __nv_bfloat16* tm = mats + c * (3 + (WANT_Y ? PP : 0)) * G::MAT;
        __nv_bfloat16* pm = tm + 3 * G::MAT;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float2 bs = pair_at(ws + BLK + c * kChunk, n, lane);
            const int s = 8 * n + 2 * (lane % 4);
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                const int t = lane / 4 + 8 * hrow;
                const float g0 = gam[t * 17 + s] * bs.x, g1 = gam[t * 17 + s + 1] * bs.y;
                amat[t * 20 + s] = s < t ? g0 * kk[n][2 * hrow] : 0.f;
                amat[t * 20 + s + 1] = s + 1 < t ? g1 * kk[n][2 * hrow + 1] : 0.f;
                if constexpr (WANT_Y) put_pieces<PP>(pm, t, s, g0 * rk[n][2 * hrow], g1 * rk[n][2 * hrow + 1]);
            }
        }
        __syncwarp();
        put_inverse(tm, amat, lane);
        __syncwarp();
    };

    const int rb_ = (lane & 7) + (lane >> 4) * 8, cb_ = ((lane >> 3) & 1) * 8;      // B operand rows, plain
    const int rt_ = (lane & 7) + ((lane >> 3) & 1) * 8, ct_ = (lane >> 4) * 8;      // B operand rows, transposed
    const uint32_t off_b = uint32_t(rb_ * LD + cb_) * 2, off_t = uint32_t(rt_ * LD + ct_) * 2;
    const uint32_t off_m = uint32_t(rb_ * kMatLd + cb_) * 2;

    fetch(0, 0);
    int st = 0;
    for (int64_t t0 = 0; t0 < a.T; t0 += BLK, st ^= 1) {
        const int nt = a.T - t0 < BLK ? int(a.T - t0) : BLK;
        const int nch = (nt + kChunk - 1) / kChunk;
        cp_async_wait();
        __syncthreads();   // the block is staged, and everyone is done with the one before
        const __nv_bfloat16* kb = ops + (KP == 1 ? st * G::OPS : 0);
        const __nv_bfloat16* rb = kb + KP * G::PIECE;
        if constexpr (KP == 3) {
            split_rows<BLK, N, G::LDR, LD, G::THREADS>(ops, G::PIECE, raw, tid);
            if constexpr (WANT_Y)
                split_rows<BLK, N, G::LDR, LD, G::THREADS>(ops + KP * G::PIECE, G::PIECE, raw + BLK * G::LDR, tid);
            __syncthreads();
        }
        if (t0 + BLK < a.T) fetch(t0 + BLK, st ^ 1);
        const float* ws = wb + st * 2 * BLK;
        for (int c = warp; c < nch; c += NW) prepare(c, kb, rb, ws);
        __syncthreads();

        IO* vb = vbuf + st * G::VEL;
#pragma unroll 1
        for (int c = 0; c < nch; ++c) {
            const uint32_t ka = smem_u32(kb + c * kChunk * LD), ra = smem_u32(rb + c * kChunk * LD);
            float pa[3][2][4] = {}, qa[PP][2][4] = {};
            // K S and R S, transposed
#pragma unroll
            for (int kk = 0; kk < N / 16; ++kk) {
                uint32_t sp[3][4];
                split_a<3>(S[2 * kk], S[2 * kk + 1], sp);
#pragma unroll
                for (int p = 0; p < KP; ++p) {
                    uint32_t f[4];
                    ldsm4(f, ka + off_b + (p * G::PIECE + kk * 16) * 2);
#pragma unroll
                    for (int i = 0; i + p < 3; ++i) {
                        mma(pa[i + p][0], sp[i], f[0], f[1]);
                        mma(pa[i + p][1], sp[i], f[2], f[3]);
                    }
                    if constexpr (WANT_Y) {
                        ldsm4(f, ra + off_b + (p * G::PIECE + kk * 16) * 2);
#pragma unroll
                        for (int i = 0; i + p < PP; ++i) {
                            mma(qa[i + p][0], sp[i], f[0], f[1]);
                            mma(qa[i + p][1], sp[i], f[2], f[3]);
                        }
                    }
                }
            }
            // X = V - g K S
            float x[2][4];
            float2 gg[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) gg[n] = pair_at(sc + c * kChunk, n, lane);
            load_lines(x, vb + c * kChunk * G::LDV + j0, G::LDV, lane);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[n][i] = fmaf(-((i & 1) ? gg[n].y : gg[n].x), pa[0][n][i] + (pa[1][n][i] + pa[2][n][i]), x[n][i]);
            // E = (I + A)^-1 X
            const __nv_bfloat16* tm = mats + c * (3 + (WANT_Y ? PP : 0)) * G::MAT;
            uint32_t xp[3][4];
            split_a<3>(x[0], x[1], xp);
            float e[2][4];
            {
                float ea[3][2][4] = {};
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    uint32_t f[4];
                    ldsm4(f, smem_u32(tm + p * G::MAT) + off_m);
#pragma unroll
                    for (int i = 0; i + p < 3; ++i) {
                        mma(ea[i + p][0], xp[i], f[0], f[1]);
                        mma(ea[i + p][1], xp[i], f[2], f[3]);
                    }
                }
                sum_orders<3>(e, ea);
            }
            // S <- g_15 S + (G beta E)^T K
            {
                float u[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float2 f = pair_at(sc + BLK + c * kChunk, n, lane);
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[n][i] = e[n][i] * ((i & 1) ? f.y : f.x);
                }
                uint32_t up[3][4];
                split_a<3>(u[0], u[1], up);
                const float gl = sc[c * kChunk + kChunk - 1];
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    float d[2][4] = {};
                    uint32_t f[KP][4];
#pragma unroll
                    for (int p = 0; p < KP; ++p) ldsm4t(f[p], ka + off_t + (p * G::PIECE + kk * 16) * 2);
#pragma unroll
                    for (int o = 2; o >= 0; --o)
#pragma unroll
                        for (int p = 0; p < KP && p <= o; ++p) {
                            mma(d[0], up[o - p], f[p][0], f[p][1]);
                            mma(d[1], up[o - p], f[p][2], f[p][3]);
                        }
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) S[2 * kk + n][i] = fmaf(gl, S[2 * kk + n][i], d[n][i]);
                }
            }
            if constexpr (!WANT_Y) {
                store_lines(a.e + vbase + (t0 + c * kChunk) * vs + j0, vs, nt - c * kChunk, e, vb, 0, false, lane);
            } else {
                // Y = g R S + P E
                uint32_t ep[PP][4];
                split_a<PP>(e[0], e[1], ep);
                float ya[PP][2][4] = {};
                const __nv_bfloat16* pm = tm + 3 * G::MAT;
#pragma unroll
                for (int p = 0; p < PP; ++p) {
                    uint32_t f[4];
                    ldsm4(f, smem_u32(pm + p * G::MAT) + off_m);
#pragma unroll
                    for (int i = 0; i + p < PP; ++i) {
                        mma(ya[i + p][0], ep[i], f[0], f[1]);
                        mma(ya[i + p][1], ep[i], f[2], f[3]);
                    }
                }
                float y[2][4], q[2][4];
                sum_orders<PP>(q, qa);
                sum_orders<PP>(y, ya);
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[n][i] = fmaf((i & 1) ? gg[n].y : gg[n].x, q[n][i], y[n][i]);
                // through the V tile's columns, which only this warp reads
                store_lines(static_cast<IO*>(a.y) + vbase + (t0 + c * kChunk) * vs + j0, vs, nt - c * kChunk, y,
                            vb + c * kChunk * G::LDV + j0, G::LDV, a.vec, lane);
            }
        }
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
