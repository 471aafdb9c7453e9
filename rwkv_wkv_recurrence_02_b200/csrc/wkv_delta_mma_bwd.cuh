// wkv_delta_mma_bwd.cuh -- reverse mode of the gated delta rule in chunks of
// 16 tokens on the tensor cores (wkv_delta_mma.cuh has the notation, the
// layouts and how float32 accuracy is kept).
//
// Within a chunk left by gradient state D (of the state after it), G[t][s]
// the decays of tokens s+1 .. t, g_t those of tokens 0 .. t, q_t those of
// tokens t+1 .. 15:
//   (I + B)^T DU = diag(q) D^T K + P^T DY,   B[s][t] = G[s][t] beta_s k_s.k_t  (t < s)
//                                            P[s][t] = G[s][t] r_s.k_t         (t <= s)
//   dv = beta du
//   D  <- g_15 D + R^T diag(g) DY - K^T diag(g beta) DU
// with the state S that enters the chunk and u = beta e:
//   dr_t = g_t S dy_t + sum_{s<=t} G[t][s] (u_s.dy_t) k_s
//   dk_t = q_t D u_t + sum_{s>=t} G[s][t] (dy_s.u_t) r_s - sum_{s>t} G[s][t] (dv_s.u_t) k_s
//          - g_t S dv_t - sum_{s<t} G[t][s] (u_s.dv_t) k_s
// Four walks: e (the forward kernel), du (value columns, backwards), the
// state's part of dr and dk (key rows), the gradient state's part of dk (key
// rows, backwards).  What only reaches dk, rounded to bfloat16, takes the
// orders up to 2^-8; dr takes them all, as r.dr enters dw.
#pragma once

#include "wkv_delta_mma.cuh"

namespace wkv {
namespace delta {

// shared-memory offsets (elements) of this lane in a B operand: rows as they
// lie (row = column of the product) and transposed (row = its k)
__device__ __forceinline__ int b_plain(int lane, int ld) { return ((lane & 7) + (lane >> 4) * 8) * ld + ((lane >> 3) & 1) * 8; }
__device__ __forceinline__ int b_trans(int lane, int ld) { return ((lane & 7) + ((lane >> 3) & 1) * 8) * ld + (lane >> 4) * 8; }

// c += A (16 x 16) B (16 x 16), NA and NB pieces, ORD orders, each in its own accumulator
template <int NA, int NB, int ORD, bool TRANS>
__device__ __forceinline__ void times(float (&c)[ORD][2][4], const uint32_t (&a)[NA][4], const __nv_bfloat16* m, int piece,
                                      int off) {
#pragma unroll
    for (int p = 0; p < NB; ++p) {
        uint32_t f[4];
        if constexpr (TRANS) ldsm4t(f, smem_u32(m + p * piece + off));
        else ldsm4(f, smem_u32(m + p * piece + off));
#pragma unroll
        for (int i = 0; i < NA && i + p < ORD; ++i) {
            mma(c[i + p][0], a[i], f[0], f[1]);
            mma(c[i + p][1], a[i], f[2], f[3]);
        }
    }
}
// the same into one accumulator, smallest orders first
template <int NA, int NB>
__device__ __forceinline__ void times_add(float (&c)[2][4], const uint32_t (&a)[NA][4], const __nv_bfloat16* m, int piece,
                                          int off) {
    uint32_t f[NB][4];
#pragma unroll
    for (int p = 0; p < NB; ++p) ldsm4t(f[p], smem_u32(m + p * piece + off));
#pragma unroll
    for (int o = 2; o >= 0; --o)
#pragma unroll
        for (int p = 0; p < NB && p <= o; ++p)
            if (o - p < NA) {
                mma(c[0], a[o - p], f[p][0], f[p][1]);
                mma(c[1], a[o - p], f[p][2], f[p][3]);
            }
}

// ---------------------------------------------------------------------------
// du, dv and the initial state's gradient (value columns)
// ---------------------------------------------------------------------------
template <typename IO, int N, int NW>
struct MmaReverse {
    static constexpr int KP = sizeof(IO) == 2 ? 1 : 3;
    static constexpr int CW = 16 * NW, SLICES = N / CW, THREADS = 32 * NW;
    static constexpr int BLK = KP == 3 && N == 128 ? 32 : 64;
    static constexpr int LD = N + 8, PIECE = BLK * LD, OPS = 2 * KP * PIECE;
    static constexpr int LDV = KP == 1 ? CW + 8 : CW + 4, VEL = BLK * LDV, LDR = N;
    static constexpr int MAT = kChunk * kMatLd, NCH = BLK / kChunk;
    static constexpr int B_OPS = OPS * 2 * (KP == 1 ? 2 : 1);
    static constexpr int B_RAW = KP == 1 ? 0 : 2 * BLK * LDR * 4;
    static constexpr int B_V = 2 * VEL * int(sizeof(IO));
    static constexpr int B_MAT = NCH * 6 * MAT * 2;
    static constexpr int B_SC = (4 + 3) * BLK * 4;
    static constexpr int B_SCR = NW * (16 * 17 + 16 * 20 + 12) * 4;
    static constexpr int SMEM = B_OPS + B_RAW + B_V + B_MAT + B_SC + B_SCR;
};

template <typename IO, int N, int NW>
__global__ void __launch_bounds__(32 * NW) delta_reverse_mma_kernel(const Args a) {
    using G = MmaReverse<IO, N, NW>;
    constexpr int KP = G::KP, LD = G::LD, NT = N / 8, BLK = G::BLK;
    extern __shared__ __align__(16) char smem_raw[];
    __nv_bfloat16* ops = reinterpret_cast<__nv_bfloat16*>(smem_raw);
    float* raw = reinterpret_cast<float*>(smem_raw + G::B_OPS);
    IO* ybuf = reinterpret_cast<IO*>(smem_raw + G::B_OPS + G::B_RAW);
    __nv_bfloat16* mats = reinterpret_cast<__nv_bfloat16*>(smem_raw + G::B_OPS + G::B_RAW + G::B_V);
    float* wb = reinterpret_cast<float*>(smem_raw + G::B_OPS + G::B_RAW + G::B_V + G::B_MAT);
    float* sc = wb + 4 * BLK;   // q, g, g beta
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    float* gam = sc + 3 * BLK + warp * (16 * 17 + 16 * 20 + 12);
    float* amat = gam + 16 * 17 + 8;

    const int64_t head = blockIdx.x / G::SLICES;
    const int slice = int(blockIdx.x % G::SLICES) * G::CW;
    const int64_t b = head / a.H, h = head % a.H, hk = h / (a.H / a.Hk);
    const int64_t ks = a.Hk * N, vs = a.H * N;
    const IO* kp = static_cast<const IO*>(a.k) + (b * a.T * a.Hk + hk) * N;
    const IO* rp = static_cast<const IO*>(a.r) + (b * a.T * a.Hk + hk) * N;
    const int64_t vbase = (b * a.T * a.H + h) * N + slice;
    const IO* yp = static_cast<const IO*>(a.dy) + vbase;
    const float* wp = a.w + b * a.T * a.H + h;
    const float* bp = a.beta + b * a.T * a.H + h;
    const int j0 = warp * 16;

    asm volatile("griddepcontrol.wait;" ::: "memory");

    float S[NT][4];   // D^T
    {
        const float* s = a.ds_out + head * N * N + slice + j0 + lane / 4;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                S[n][i] = a.ds_out != nullptr ? s[(8 * n + 2 * (lane % 4) + (i & 1)) * N + (i >> 1) * 8] : 0.f;
    }

    auto fetch = [&](int64_t t0, int st) {
        const int nt = a.T - t0 < BLK ? int(a.T - t0) : BLK;
        if constexpr (KP == 1) {
            copy_rows<IO, BLK, N, LD, G::THREADS>(reinterpret_cast<IO*>(ops + st * G::OPS), kp + t0 * ks, ks, nt, a.vec, tid);
            copy_rows<IO, BLK, N, LD, G::THREADS>(reinterpret_cast<IO*>(ops + st * G::OPS + G::PIECE), rp + t0 * ks, ks, nt,
                                                  a.vec, tid);
        } else {
            copy_rows<float, BLK, N, G::LDR, G::THREADS>(raw, reinterpret_cast<const float*>(kp) + t0 * ks, ks, nt, a.vec, tid);
            copy_rows<float, BLK, N, G::LDR, G::THREADS>(raw + BLK * G::LDR, reinterpret_cast<const float*>(rp) + t0 * ks, ks,
                                                         nt, a.vec, tid);
        }
        copy_rows<IO, BLK, G::CW, G::LDV, G::THREADS>(ybuf + st * G::VEL, yp + t0 * vs, vs, nt, a.vec, tid);
        for (int t = tid; t < BLK; t += G::THREADS) {
            wb[st * 2 * BLK + t] = t < nt ? wp[(t0 + t) * a.H] : 0.f;
            wb[(st * 2 + 1) * BLK + t] = t < nt ? bp[(t0 + t) * a.H] : 0.f;
        }
        cp_async_commit();
    };

    auto prepare = [&](int c, const __nv_bfloat16* kb, const __nv_bfloat16* rb, const float* ws) {
        const int tl = lane % 16;
        const ChunkDecay d = chunk_decay(ws + c * kChunk, gam, lane);
        if (lane < 16) {
            sc[c * kChunk + tl] = d.after;
            sc[BLK + c * kChunk + tl] = d.upto;
            sc[2 * BLK + c * kChunk + tl] = d.upto * ws[BLK + c * kChunk + tl];
        }
        __syncwarp();
        float kk[2][4], rk[2][4];
        gram<N, KP, KP, KP>(kk, kb + c * kChunk * LD, kb + c * kChunk * LD, G::PIECE, lane);
        gram<N, KP, KP, KP>(rk, rb + c * kChunk * LD, kb + c * kChunk * LD, G::PIECE, lane);
        __nv_bfloat16* tm = mats + c * 6 * G::MAT;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int t = 8 * n + 2 * (lane % 4);
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                const int s = lane / 4 + 8 * hrow;
                const float bs = ws[BLK + c * kChunk + s];
                const float g0 = gam[s * 17 + t], g1 = gam[s * 17 + t + 1];
                amat[s * 20 + t] = t < s ? g0 * bs * kk[n][2 * hrow] : 0.f;
                amat[s * 20 + t + 1] = t + 1 < s ? g1 * bs * kk[n][2 * hrow + 1] : 0.f;
                put_pieces<3>(tm + 3 * G::MAT, s, t, g0 * rk[n][2 * hrow], g1 * rk[n][2 * hrow + 1]);
            }
        }
        __syncwarp();
        put_inverse(tm, amat, lane);
        __syncwarp();
    };

    const int off_b = b_plain(lane, LD), off_t = b_trans(lane, LD), off_m = b_trans(lane, kMatLd);
    const int64_t last = (a.T - 1) / BLK * BLK;
    fetch(last, 0);
    int st = 0;
    for (int64_t t0 = last; t0 >= 0; t0 -= BLK, st ^= 1) {
        const int nt = a.T - t0 < BLK ? int(a.T - t0) : BLK;
        const int nch = (nt + kChunk - 1) / kChunk;
        cp_async_wait();
        __syncthreads();
        const __nv_bfloat16* kb = ops + (KP == 1 ? st * G::OPS : 0);
        const __nv_bfloat16* rb = kb + KP * G::PIECE;
        if constexpr (KP == 3) {
            split_rows<BLK, N, G::LDR, LD, G::THREADS>(ops, G::PIECE, raw, tid);
            split_rows<BLK, N, G::LDR, LD, G::THREADS>(ops + KP * G::PIECE, G::PIECE, raw + BLK * G::LDR, tid);
            __syncthreads();
        }
        if (t0 > 0) fetch(t0 - BLK, st ^ 1);
        const float* ws = wb + st * 2 * BLK;
        for (int c = warp; c < nch; c += NW) prepare(c, kb, rb, ws);
        __syncthreads();

        IO* yb = ybuf + st * G::VEL;
#pragma unroll 1
        for (int c = nch - 1; c >= 0; --c) {
            const __nv_bfloat16* kc = kb + c * kChunk * LD;
            const __nv_bfloat16* rc = rb + c * kChunk * LD;
            const __nv_bfloat16* tm = mats + c * 6 * G::MAT;
            float dy[2][4], x[2][4];
            {
                float pa[3][2][4] = {};
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    uint32_t sp[3][4];
                    split_a<3>(S[2 * kk], S[2 * kk + 1], sp);
                    times<3, KP, 3, false>(pa, sp, kc + kk * 16, G::PIECE, off_b);
                }
                sum_orders<3>(x, pa);
                scale_tokens(x, sc + c * kChunk, lane);
            }
            load_lines(dy, yb + c * kChunk * G::LDV + j0, G::LDV, lane);
            {
                uint32_t yq[KP][4];
                split_a<KP>(dy[0], dy[1], yq);
                float ya[3][2][4] = {};
                times<KP, 3, 3, true>(ya, yq, tm + 3 * G::MAT, G::MAT, off_m);
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[n][i] += ya[0][n][i] + (ya[1][n][i] + ya[2][n][i]);
            }
            float du[2][4];
            {
                uint32_t xp[3][4];
                split_a<3>(x[0], x[1], xp);
                float ea[3][2][4] = {};
                times<3, 3, 3, true>(ea, xp, tm, G::MAT, off_m);
                sum_orders<3>(du, ea);
            }
            // D <- g_15 D + (g dy)^T R - (g beta du)^T K
            {
                float f0[2][4], f1[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) f0[n][i] = dy[n][i], f1[n][i] = -du[n][i];
                scale_tokens(f0, sc + BLK + c * kChunk, lane);
                scale_tokens(f1, sc + 2 * BLK + c * kChunk, lane);
                uint32_t yq[3][4], uq[3][4];
                split_a<3>(f0[0], f0[1], yq);
                split_a<3>(f1[0], f1[1], uq);
                const float gl = sc[BLK + c * kChunk + kChunk - 1];
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    float d[2][4] = {};
                    times_add<3, KP>(d, uq, kc + kk * 16, G::PIECE, off_t);
                    times_add<3, KP>(d, yq, rc + kk * 16, G::PIECE, off_t);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) S[2 * kk + n][i] = fmaf(gl, S[2 * kk + n][i], d[n][i]);
                }
            }
            const int64_t at = vbase + (t0 + c * kChunk) * vs + j0;
            store_lines(a.du + at, vs, nt - c * kChunk, du, yb, 0, false, lane);
            scale_tokens(du, ws + BLK + c * kChunk, lane);
            // dv through dy's columns, which only this warp reads
            store_lines(static_cast<IO*>(a.dv) + at, vs, nt - c * kChunk, du, yb + c * kChunk * G::LDV + j0, G::LDV, a.vec, lane);
        }
    }
    if (a.ds_in != nullptr) {
        float* s = a.ds_in + head * N * N + slice + j0 + lane / 4;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[(8 * n + 2 * (lane % 4) + (i & 1)) * N + (i >> 1) * 8] = S[n][i];
    }
}

// ---------------------------------------------------------------------------
// Key rows: a warp owns 16 key rows of S (or D) for the whole value axis.
// GRAD false: the state's walk forwards -- dr, the state's part of dk, and
// the states at the borders of kCheck tokens.  GRAD true: the gradient
// state's walk backwards -- its part of dk and the border products <D, S>.
// ---------------------------------------------------------------------------
template <typename IO, int N, int NW, bool GRAD>
struct MmaRows {
    static constexpr int KP = sizeof(IO) == 2 ? 1 : 3;
    static constexpr int PP = sizeof(IO) == 2 ? 2 : 3;   // orders of what only reaches dk
    static constexpr int KE = GRAD ? PP : 3, KD = GRAD ? 3 : PP;   // pieces of e and du
    static constexpr int CW = 16 * NW, SLICES = N / CW, THREADS = 32 * NW, SLOTS = N / 16;
    static constexpr int BLK = 32;
    static constexpr int LD = N + 8, PIECE = BLK * LD, LDR = N, ROW = BLK * LDR;
    static constexpr int LDV = KP == 1 ? CW + 8 : CW + 4, VEL = BLK * LDV;
    static constexpr int MAT = kChunk * kMatLd, NCH = BLK / kChunk;
    static constexpr int M0 = PP, M1 = GRAD ? PP : 3;    // pieces of the two 16 x 16 matrices
    static constexpr int OPS = KE + KD + KP * (KP == 1 ? 2 : 1);   // staged arrays of PIECE elements
    static constexpr int B_OPS = OPS * PIECE * 2;
    static constexpr int B_RAW = (KP == 1 ? 2 : 3) * ROW * 4;
    static constexpr int B_V = 2 * (GRAD ? 2 : 1) * VEL * int(sizeof(IO));
    static constexpr int B_MAT = NCH * (M0 + M1) * MAT * 2;
    static constexpr int B_SC = (4 + 4) * BLK * 4;
    static constexpr int B_SCR = NW * (16 * 17) * 4;
    static constexpr int SMEM = B_OPS + B_RAW + B_V + B_MAT + B_SC + B_SCR;
};

// float32 rows as NP bfloat16 pieces
template <int BLK, int W, int LDS, int LDD, int NP, int THREADS>
__device__ __forceinline__ void split_rows_np(__nv_bfloat16* dst, int piece, const float* src, int tid) {
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

template <typename IO, int N, int NW, bool GRAD>
__global__ void __launch_bounds__(32 * NW) delta_rows_mma_kernel(const Args a) {
    using G = MmaRows<IO, N, NW, GRAD>;
    constexpr int KP = G::KP, PP = G::PP, KE = G::KE, KD = G::KD, LD = G::LD, NT = N / 8, BLK = G::BLK;
    extern __shared__ __align__(16) char smem_raw[];
    __nv_bfloat16* eb = reinterpret_cast<__nv_bfloat16*>(smem_raw);
    __nv_bfloat16* db = eb + KE * G::PIECE;
    __nv_bfloat16* yops = db + KD * G::PIECE;
    float* raw = reinterpret_cast<float*>(smem_raw + G::B_OPS);   // e, du (, dy)
    IO* slices = reinterpret_cast<IO*>(smem_raw + G::B_OPS + G::B_RAW);   // k (and r) of the CTA's rows, two stages
    __nv_bfloat16* mats = reinterpret_cast<__nv_bfloat16*>(smem_raw + G::B_OPS + G::B_RAW + G::B_V);
    float* wb = reinterpret_cast<float*>(smem_raw + G::B_OPS + G::B_RAW + G::B_V + G::B_MAT);
    float* sc = wb + 4 * BLK;   // g, g beta, q beta, -
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    float* gam = sc + 4 * BLK + warp * (16 * 17);

    const int64_t head = blockIdx.x / G::SLICES;
    const int slice = int(blockIdx.x % G::SLICES) * G::CW;
    const int64_t b = head / a.H, h = head % a.H, hk = h / (a.H / a.Hk);
    const int64_t ks = a.Hk * N, vs = a.H * N;
    const int64_t base = (b * a.T * a.H + h) * N;
    const IO* kp = static_cast<const IO*>(a.k) + (b * a.T * a.Hk + hk) * N + slice;
    const IO* rp = static_cast<const IO*>(a.r) + (b * a.T * a.Hk + hk) * N + slice;
    const IO* yp = static_cast<const IO*>(a.dy) + base;
    const float* wp = a.w + b * a.T * a.H + h;
    const float* bp = a.beta + b * a.T * a.H + h;
    const int i0 = warp * 16;
    const int64_t nchunk = (a.T + kCheck - 1) / kCheck;
    const int slot = slice / 16 + warp;
    float* ck = a.check + head * (nchunk + 1) * N * N + slot * (N * 16);
    float* phi = a.phi + head * (nchunk + 1) * G::SLOTS + slot;

    asm volatile("griddepcontrol.wait;" ::: "memory");

    // tile n: values 8 n .. 8 n + 7 of key rows i0 + lane / 4 (+ 8)
    float S[NT][4];
    const float* s0 = GRAD ? a.ds_out : a.s_in;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            S[n][i] = s0 != nullptr ? s0[head * N * N + (slice + i0 + lane / 4 + (i >> 1) * 8) * N + 8 * n + 2 * (lane % 4) + (i & 1)]
                                    : 0.f;
    auto keep = [&](int64_t c) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
            reinterpret_cast<float4*>(ck + c * N * N)[n * 32 + lane] = make_float4(S[n][0], S[n][1], S[n][2], S[n][3]);
    };
    auto border = [&](int64_t c) {
        float x = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(ck + c * N * N) + n * 32 + lane);
            x = fmaf(S[n][0], v.x, x);
            x = fmaf(S[n][1], v.y, x);
            x = fmaf(S[n][2], v.z, x);
            x = fmaf(S[n][3], v.w, x);
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) phi[c * G::SLOTS] = x;
    };
    if constexpr (GRAD) {
        if (s0 != nullptr) border(nchunk);
        else if (lane == 0) phi[nchunk * G::SLOTS] = 0.f;
    }

    auto fetch = [&](int64_t t0, int st) {
        const int nt = a.T - t0 < BLK ? int(a.T - t0) : BLK;
        copy_rows<float, BLK, N, G::LDR, G::THREADS>(raw, a.e + base + t0 * vs, vs, nt, true, tid);
        copy_rows<float, BLK, N, G::LDR, G::THREADS>(raw + G::ROW, a.du + base + t0 * vs, vs, nt, true, tid);
        if constexpr (KP == 1)
            copy_rows<IO, BLK, N, LD, G::THREADS>(reinterpret_cast<IO*>(yops + st * G::PIECE), yp + t0 * vs, vs, nt, a.vec, tid);
        else
            copy_rows<float, BLK, N, G::LDR, G::THREADS>(raw + 2 * G::ROW, reinterpret_cast<const float*>(yp) + t0 * vs, vs, nt,
                                                         a.vec, tid);
        IO* sl = slices + st * (GRAD ? 2 : 1) * G::VEL;
        copy_rows<IO, BLK, G::CW, G::LDV, G::THREADS>(sl, kp + t0 * ks, ks, nt, a.vec, tid);
        if constexpr (GRAD) copy_rows<IO, BLK, G::CW, G::LDV, G::THREADS>(sl + G::VEL, rp + t0 * ks, ks, nt, a.vec, tid);
        for (int t = tid; t < BLK; t += G::THREADS) {
            wb[st * 2 * BLK + t] = t < nt ? wp[(t0 + t) * a.H] : 0.f;
            wb[(st * 2 + 1) * BLK + t] = t < nt ? bp[(t0 + t) * a.H] : 0.f;
        }
        cp_async_commit();
    };

    // one of the two matrices of a chunk (one warp)
    auto prepare = [&](int c, int which, const __nv_bfloat16* yb, const float* ws) {
        const int tl = lane % 16;
        const float* be = ws + BLK + c * kChunk;
        const ChunkDecay d = chunk_decay(ws + c * kChunk, gam, lane);
        if (which == 0 && lane < 16) {
            sc[c * kChunk + tl] = d.upto;
            sc[BLK + c * kChunk + tl] = d.upto * be[tl];
            sc[2 * BLK + c * kChunk + tl] = d.after * be[tl];
        }
        __syncwarp();
        const __nv_bfloat16 *ec = eb + c * kChunk * LD, *dc = db + c * kChunk * LD, *yc = yb + c * kChunk * LD;
        __nv_bfloat16* m = mats + (c * (G::M0 + G::M1) + (which ? G::M0 : 0)) * G::MAT;
        float x[2][4];
        if constexpr (!GRAD) {
            // which 0: G[t][s] beta_s beta_t e_s.du_t (s < t); 1: G[t][s] beta_s e_s.dy_t (s <= t)
            if (which == 0) gram<N, KD, KE, PP>(x, dc, ec, G::PIECE, lane);
            else gram<N, KP, KE, 3>(x, yc, ec, G::PIECE, lane);
        } else {
            // which 0: G[s][t] beta_t e_t.dy_s (s >= t); 1: -G[s][t] beta_s beta_t e_t.du_s (s > t)
            if (which == 0) gram<N, KE, KP, PP>(x, ec, yc, G::PIECE, lane);
            else gram<N, KE, PP, PP>(x, ec, dc, G::PIECE, lane);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                const int t = lane / 4 + 8 * hrow;
                float v[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int s = 8 * n + 2 * (lane % 4) + q;
                    const float g = GRAD ? gam[s * 17 + t] : gam[t * 17 + s];
                    float f;
                    if constexpr (!GRAD) f = which == 0 ? (s < t ? g * be[s] * be[t] : 0.f) : g * be[s];
                    else f = which == 0 ? g * be[t] : (s > t ? -g * be[s] * be[t] : 0.f);
                    v[q] = f * x[n][2 * hrow + q];
                }
                const int s = 8 * n + 2 * (lane % 4);
                if (which == 0) put_pieces<G::M0>(m, t, s, v[0], v[1]);
                else put_pieces<G::M1>(m, t, s, v[0], v[1]);
            }
        __syncwarp();
    };

    const int off_b = b_plain(lane, LD), off_t = b_trans(lane, LD), off_m = b_plain(lane, kMatLd);
    const int64_t last = (a.T - 1) / BLK * BLK;
    fetch(GRAD ? last : 0, 0);
    int st = 0;
    for (int64_t t0 = GRAD ? last : 0; GRAD ? t0 >= 0 : t0 < a.T; t0 += GRAD ? -BLK : BLK, st ^= 1) {
        const int nt = a.T - t0 < BLK ? int(a.T - t0) : BLK;
        const int nch = (nt + kChunk - 1) / kChunk;
        cp_async_wait();
        __syncthreads();
        split_rows_np<BLK, N, G::LDR, LD, KE, G::THREADS>(eb, G::PIECE, raw, tid);
        split_rows_np<BLK, N, G::LDR, LD, KD, G::THREADS>(db, G::PIECE, raw + G::ROW, tid);
        if constexpr (KP == 3) split_rows_np<BLK, N, G::LDR, LD, 3, G::THREADS>(yops, G::PIECE, raw + 2 * G::ROW, tid);
        __syncthreads();
        if (GRAD ? t0 > 0 : t0 + BLK < a.T) fetch(GRAD ? t0 - BLK : t0 + BLK, st ^ 1);
        const __nv_bfloat16* yb = yops + (KP == 1 ? st * G::PIECE : 0);
        const float* ws = wb + st * 2 * BLK;
        for (int i = warp; i < 2 * nch; i += NW) prepare(i / 2, i % 2, yb, ws);
        if constexpr (!GRAD) {
            if (t0 % kCheck == 0) keep(t0 / kCheck);
        }
        __syncthreads();

        IO* kt = slices + st * (GRAD ? 2 : 1) * G::VEL;
#pragma unroll 1
        for (int cc = 0; cc < nch; ++cc) {
            const int c = GRAD ? nch - 1 - cc : cc;
            const __nv_bfloat16 *ec = eb + c * kChunk * LD, *dc = db + c * kChunk * LD, *yc = yb + c * kChunk * LD;
            const __nv_bfloat16* m0 = mats + c * (G::M0 + G::M1) * G::MAT;
            const __nv_bfloat16* m1 = m0 + G::M0 * G::MAT;
            const int64_t at = base + (t0 + c * kChunk) * vs + slice + i0;
            const int left = nt - c * kChunk;
            float k[2][4];
            load_lines(k, kt + c * kChunk * G::LDV + i0, G::LDV, lane);
            uint32_t kq[KP][4];
            split_a<KP>(k[0], k[1], kq);
            const float gl = sc[c * kChunk + kChunk - 1];
            if constexpr (!GRAD) {
                float o1[2][4], o2[2][4];
                {
                    float pa[PP][2][4] = {}, qa[3][2][4] = {};
#pragma unroll
                    for (int kk = 0; kk < N / 16; ++kk) {
                        uint32_t sp[3][4];
                        split_a<3>(S[2 * kk], S[2 * kk + 1], sp);
                        times<3, KD, PP, false>(pa, sp, dc + kk * 16, G::PIECE, off_b);
                        times<3, KP, 3, false>(qa, sp, yc + kk * 16, G::PIECE, off_b);
                    }
                    sum_orders<PP>(o1, pa);
                    sum_orders<3>(o2, qa);
                    scale_tokens(o1, sc + BLK + c * kChunk, lane);
                    scale_tokens(o2, sc + c * kChunk, lane);
                }
                {
                    float pa[PP][2][4] = {}, qa[3][2][4] = {};
                    times<KP, G::M0, PP, false>(pa, kq, m0, G::MAT, off_m);
                    times<KP, G::M1, 3, false>(qa, kq, m1, G::MAT, off_m);
                    float p[2][4], q[2][4];
                    sum_orders<PP>(p, pa);
                    sum_orders<3>(q, qa);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o1[n][i] = -(o1[n][i] + p[n][i]), o2[n][i] += q[n][i];
                }
                // S <- g_15 S + (G beta k) e^T
                scale_tokens(k, sc + 2 * BLK + c * kChunk, lane);
                uint32_t ks3[3][4];
                split_a<3>(k[0], k[1], ks3);
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    float d[2][4] = {};
                    times_add<3, 3>(d, ks3, ec + kk * 16, G::PIECE, off_t);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) S[2 * kk + n][i] = fmaf(gl, S[2 * kk + n][i], d[n][i]);
                }
                store_lines(a.dk + at, vs, left, o1, kt, 0, false, lane);
                store_lines(a.dr + at, vs, left, o2, kt, 0, false, lane);
            } else {
                float r[2][4];
                load_lines(r, kt + G::VEL + c * kChunk * G::LDV + i0, G::LDV, lane);
                uint32_t rq[KP][4];
                split_a<KP>(r[0], r[1], rq);
                float o[2][4];
                {
                    float pa[PP][2][4] = {};
#pragma unroll
                    for (int kk = 0; kk < N / 16; ++kk) {
                        uint32_t sp[PP][4];
                        split_a<PP>(S[2 * kk], S[2 * kk + 1], sp);
                        times<PP, KE, PP, false>(pa, sp, ec + kk * 16, G::PIECE, off_b);
                    }
                    sum_orders<PP>(o, pa);
                    scale_tokens(o, sc + 2 * BLK + c * kChunk, lane);
                }
                {
                    float pa[PP][2][4] = {};
                    times<KP, G::M0, PP, false>(pa, rq, m0, G::MAT, off_m);
                    times<KP, G::M1, PP, false>(pa, kq, m1, G::MAT, off_m);
                    float p[2][4];
                    sum_orders<PP>(p, pa);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[n][i] += p[n][i], k[n][i] = -k[n][i];
                }
                // D <- g_15 D + (g r) dy^T - (g beta k) du^T
                scale_tokens(r, sc + c * kChunk, lane);
                scale_tokens(k, sc + BLK + c * kChunk, lane);
                uint32_t r3[3][4], k3[3][4];
                split_a<3>(r[0], r[1], r3);
                split_a<3>(k[0], k[1], k3);
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    float d[2][4] = {};
                    times_add<3, 3>(d, k3, dc + kk * 16, G::PIECE, off_t);
                    times_add<3, KP>(d, r3, yc + kk * 16, G::PIECE, off_t);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) S[2 * kk + n][i] = fmaf(gl, S[2 * kk + n][i], d[n][i]);
                }
                store_lines(a.dk2 + at, vs, left, o, kt, 0, false, lane);
            }
        }
        if constexpr (GRAD) {
            if (t0 % kCheck == 0) border(t0 / kCheck);
        }
    }
    if constexpr (!GRAD) keep(nchunk);
}

}  // namespace delta
}  // namespace wkv
