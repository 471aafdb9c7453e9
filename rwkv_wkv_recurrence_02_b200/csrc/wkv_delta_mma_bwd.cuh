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

// ---------------------------------------------------------------------------
// du, dv, the initial state's gradient, and dv.v for dw (value columns)
// ---------------------------------------------------------------------------
template <typename IO, int N, int NW>
using ReverseShape = MmaColumns<IO, N, NW, true, 6, 3, 2>;

template <typename IO, int N, int NW>
__global__ void __launch_bounds__(ReverseShape<IO, N, NW>::THREADS, N == 64 && sizeof(IO) == 2 ? 2 : 1)
delta_reverse_mma_kernel(const Args a) {
    using G = ReverseShape<IO, N, NW>;
    constexpr int KP = G::KP, LD = G::LD, NT = N / 8, BLK = G::BLK;
    extern __shared__ __align__(16) char smem[];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;

    const int64_t head = blockIdx.x / G::SLICES;
    const int slice = int(blockIdx.x % G::SLICES) * G::CW;
    const int64_t b = head / a.H, h = head % a.H, hk = h / (a.H / a.Hk);
    const int64_t vs = a.H * N;
    const int64_t vbase = (b * a.T * a.H + h) * N + slice;
    const int64_t last = (a.T - 1) / BLK * BLK;

    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp >= NW) {
        const int64_t ks = a.Hk * N;
        const IO* kp = static_cast<const IO*>(a.k) + (b * a.T * a.Hk + hk) * N;
        const IO* rp = static_cast<const IO*>(a.r) + (b * a.T * a.Hk + hk) * N;
        const int tl = lane % 16;
        int st = 0;
        for (int64_t t0 = last; t0 >= 0; t0 -= BLK, st ^= 1) {
            const int nt = a.T - t0 < BLK ? int(a.T - t0) : BLK;
            G g(smem, st);
            if (last - t0 >= 2 * BLK) bar_sync<G::THREADS>(kBarFree + st);
            g.fetch(smem, kp, rp, ks, static_cast<const IO*>(a.dy) + vbase, static_cast<const IO*>(a.v) + vbase, vs,
                    a.w + b * a.T * a.H + h, a.beta + b * a.T * a.H + h, a.H, t0, nt, a.vec, tid - G::WALK);
            float* gam = g.scratch(smem, warp - NW);
            float* amat = gam + 16 * 17 + 8;
            // B, its inverse and P
            for (int c = warp - NW; c * kChunk < nt; c += G::STAGERS / 32) {
                const ChunkDecay d = chunk_decay(g.w + c * kChunk, gam, lane);
                if (lane < 16) {
                    g.sc[c * kChunk + tl] = d.after;
                    g.sc[BLK + c * kChunk + tl] = d.upto;
                    g.sc[2 * BLK + c * kChunk + tl] = d.upto * g.beta[c * kChunk + tl];
                }
                __syncwarp();
                const __nv_bfloat16* kc = g.k + c * kChunk * LD;
                float kk[2][4], rk[2][4];
                gram<N, KP, KP, KP>(kk, kc, kc, G::PIECE, lane);
                gram<N, KP, KP, KP>(rk, g.r() + c * kChunk * LD, kc, G::PIECE, lane);
                __nv_bfloat16* tm = g.mats + c * 6 * G::MAT;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int t = 8 * n + 2 * (lane % 4);
#pragma unroll
                    for (int hrow = 0; hrow < 2; ++hrow) {
                        const int s = lane / 4 + 8 * hrow;
                        const float bs = g.beta[c * kChunk + s];
                        const float g0 = gam[s * 17 + t], g1 = gam[s * 17 + t + 1];
                        amat[s * 20 + t] = t < s ? g0 * bs * kk[n][2 * hrow] : 0.f;
                        amat[s * 20 + t + 1] = t + 1 < s ? g1 * bs * kk[n][2 * hrow + 1] : 0.f;
                        put_pieces<3>(tm + 3 * G::MAT, s, t, g0 * rk[n][2 * hrow], g1 * rk[n][2 * hrow + 1]);
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
    float S[NT][4];   // D^T
    {
        const float* s = a.ds_out + head * N * N + slice + j0 + lane / 4;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                S[n][i] = a.ds_out != nullptr ? s[(8 * n + 2 * (lane % 4) + (i & 1)) * N + (i >> 1) * 8] : 0.f;
    }
    float* pv = a.pv + (slice / 16 + warp) * (a.B * a.T * a.H) + b * a.T * a.H + h;
    const int off_b = b_plain(lane, LD), off_t = b_trans(lane, LD), off_m = b_trans(lane, kMatLd);
    int st = 0;
    for (int64_t t0 = last; t0 >= 0; t0 -= BLK, st ^= 1) {
        const int nt = a.T - t0 < BLK ? int(a.T - t0) : BLK;
        G g(smem, st);
        bar_sync<G::THREADS>(kBarFull + st);
#pragma unroll 1
        for (int c = (nt - 1) / kChunk; c >= 0; --c) {
            const __nv_bfloat16* kc = g.k + c * kChunk * LD;
            const __nv_bfloat16* rc = g.r() + c * kChunk * LD;
            const __nv_bfloat16* tm = g.mats + c * 6 * G::MAT;
            const float* sc = g.sc + c * kChunk;
            IO* yt = g.v + c * kChunk * G::LDV + j0;
            // diag(q) D^T K + P^T dY
            float dy[2][4], x[2][4];
            {
                Acc pa;
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    uint32_t sp[3][4];
                    split_a<3>(S[2 * kk], S[2 * kk + 1], sp);
                    times<3, KP, 3, false>(pa, kk == 0, sp, kc + kk * 16, G::PIECE, off_b);
                }
                pa.sum(x);
                scale_tokens(x, sc, lane);
            }
            load_lines(dy, yt, G::LDV, lane);
            {
                uint32_t yq[KP][4];
                split_a<KP>(dy[0], dy[1], yq);
                Acc ya;
                times<KP, 3, 3, true>(ya, true, yq, tm + 3 * G::MAT, G::MAT, off_m);
                float p[2][4];
                ya.sum(p);
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[n][i] += p[n][i];
            }
            float du[2][4];
            {
                uint32_t xp[3][4];
                split_a<3>(x[0], x[1], xp);
                Acc ea;
                times<3, 3, 3, true>(ea, true, xp, tm, G::MAT, off_m);
                ea.sum(du);
            }
            // D <- g_15 D + (g dy)^T R - (g beta du)^T K
            {
                float f1[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) f1[n][i] = -du[n][i];
                scale_tokens(dy, sc + BLK, lane);
                scale_tokens(f1, sc + 2 * BLK, lane);
                uint32_t yq[3][4], uq[3][4];
                split_a<3>(dy[0], dy[1], yq);
                split_a<3>(f1[0], f1[1], uq);
                const float gl = sc[BLK + kChunk - 1];
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    float d[2][4];
                    times_add<3, KP>(d, true, uq, kc + kk * 16, G::PIECE, off_t);
                    times_add<3, KP>(d, false, yq, rc + kk * 16, G::PIECE, off_t);
                    fade_add(S[2 * kk], gl, d[0]);
                    fade_add(S[2 * kk + 1], gl, d[1]);
                }
            }
            const int64_t t = t0 + c * kChunk, at = vbase + t * vs + j0;
            const int left = nt - c * kChunk;
            store_lines(a.du + at, vs, left, du, yt, 0, false, lane);
            scale_tokens(du, g.beta + c * kChunk, lane);
            float v[2][4];
            load_lines(v, yt + G::VEL, G::LDV, lane);
            token_sums(pv + t * a.H, a.H, left, du, v, lane);
            // dv through dy's columns, which only this warp reads
            store_lines(static_cast<IO*>(a.dv) + at, vs, left, du, yt, G::LDV, a.vec, lane);
        }
        if (t0 >= 2 * BLK) bar_arrive<G::THREADS>(kBarFree + st);
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
// GRAD false: the state's walk forwards -- dr, the state's part of dk, dbeta,
// r.dr for dw and the states at the borders of kCheck tokens.  GRAD true: the
// gradient state's walk backwards -- the rest of dk and the border products
// <D, S>.  dr and dk are final where no heads share a key head; otherwise the
// value heads' own go to the workspace.
// ---------------------------------------------------------------------------
template <typename IO, int N, int NW, bool GRAD>
struct MmaRows {
    static constexpr int KP = sizeof(IO) == 2 ? 1 : 3;
    static constexpr int PP = kOutOrders<IO>;                      // orders of what only reaches dk
    static constexpr int KE = GRAD ? PP : 3, KD = GRAD ? 3 : PP;   // pieces of e and du
    static constexpr int CW = 16 * NW, SLICES = N / CW, SLOTS = N / 16;
    static constexpr int WALK = 32 * NW, STAGERS = 64, THREADS = WALK + STAGERS;
    static constexpr int BLK = KP == 3 && N == 128 ? 16 : 32;      // what two stages leave room for
    static constexpr int LD = N + 8, PIECE = BLK * LD, LDR = N, ROW = BLK * LDR;
    static constexpr int LDV = KP == 1 ? CW + 8 : CW + 4, VEL = BLK * LDV;
    static constexpr int MAT = kChunk * kMatLd, NCH = BLK / kChunk;
    static constexpr int M0 = PP, M1 = GRAD ? PP : 3;              // pieces of the two 16 x 16 matrices
    // bytes of a stage, in order: e, du, dy; k and r of the CTA's rows; matrices; w, beta, factors
    static constexpr int S_OPS = (KE + KD + KP) * PIECE * 2, S_V = 2 * VEL * int(sizeof(IO));
    static constexpr int S_MAT = NCH * (M0 + M1) * MAT * 2, S_SC = 5 * BLK * 4;
    static constexpr int STAGE = S_OPS + S_V + S_MAT + S_SC;
    static constexpr int B_RAW = (KP == 1 ? 2 : 3) * ROW * 4;      // e, du (, dy) as they come
    static constexpr int SCR = 16 * 17;
    static constexpr int SMEM = 2 * STAGE + B_RAW + STAGERS / 32 * SCR * 4;

    __nv_bfloat16 *e, *du, *dy, *mats;
    IO *k, *r;
    float *w, *beta, *sc, *raw;
    __device__ __forceinline__ MmaRows(char* smem, int st) {
        char* p = smem + st * STAGE;
        e = reinterpret_cast<__nv_bfloat16*>(p);
        du = e + KE * PIECE;
        dy = du + KD * PIECE;
        k = reinterpret_cast<IO*>(p + S_OPS);
        r = k + VEL;
        mats = reinterpret_cast<__nv_bfloat16*>(p + S_OPS + S_V);
        w = reinterpret_cast<float*>(p + S_OPS + S_V + S_MAT);
        beta = w + BLK;
        sc = w + 2 * BLK;
        raw = reinterpret_cast<float*>(smem + 2 * STAGE);
    }
};

template <typename IO, int N, int NW, bool GRAD>
__global__ void __launch_bounds__(MmaRows<IO, N, NW, GRAD>::THREADS, N == 64 && sizeof(IO) == 2 ? 2 : 1)
delta_rows_mma_kernel(const Args a) {
    using G = MmaRows<IO, N, NW, GRAD>;
    constexpr int KP = G::KP, PP = G::PP, KE = G::KE, KD = G::KD, LD = G::LD, NT = N / 8, BLK = G::BLK;
    extern __shared__ __align__(16) char smem[];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;

    const int64_t head = blockIdx.x / G::SLICES;
    const int slice = int(blockIdx.x % G::SLICES) * G::CW;
    const int64_t b = head / a.H, h = head % a.H, hk = h / (a.H / a.Hk);
    const int64_t ks = a.Hk * N, vs = a.H * N;
    const int64_t base = (b * a.T * a.H + h) * N, scalar = b * a.T * a.H + h;
    const int64_t last = (a.T - 1) / BLK * BLK;
    const int64_t first = GRAD ? last : 0, step = GRAD ? -BLK : BLK;
    const int64_t blocks = last / BLK + 1;

    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp >= NW) {
        const int stid = tid - G::WALK, tl = lane % 16;
        const IO* kp = static_cast<const IO*>(a.k) + (b * a.T * a.Hk + hk) * N + slice;
        const IO* rp = static_cast<const IO*>(a.r) + (b * a.T * a.Hk + hk) * N + slice;
        const IO* yp = static_cast<const IO*>(a.dy) + base;
        int st = 0;
        int64_t t0 = first;
        for (int64_t i = 0; i < blocks; ++i, t0 += step, st ^= 1) {
            const int nt = a.T - t0 < BLK ? int(a.T - t0) : BLK;
            G g(smem, st);
            // the raw rows are the stagers' own; the stage is the walkers' until they leave it
            copy_rows<float, BLK, N, G::LDR, G::STAGERS>(g.raw, a.e + base + t0 * vs, vs, nt, true, stid);
            copy_rows<float, BLK, N, G::LDR, G::STAGERS>(g.raw + G::ROW, a.du + base + t0 * vs, vs, nt, true, stid);
            if constexpr (KP == 3)
                copy_rows<float, BLK, N, G::LDR, G::STAGERS>(g.raw + 2 * G::ROW, reinterpret_cast<const float*>(yp) + t0 * vs,
                                                             vs, nt, a.vec, stid);
            if (i >= 2) bar_sync<G::THREADS>(kBarFree + st);
            if constexpr (KP == 1)
                copy_rows<IO, BLK, N, LD, G::STAGERS>(reinterpret_cast<IO*>(g.dy), yp + t0 * vs, vs, nt, a.vec, stid);
            copy_rows<IO, BLK, G::CW, G::LDV, G::STAGERS>(g.k, kp + t0 * ks, ks, nt, a.vec, stid);
            copy_rows<IO, BLK, G::CW, G::LDV, G::STAGERS>(g.r, rp + t0 * ks, ks, nt, a.vec, stid);
            for (int t = stid; t < BLK; t += G::STAGERS) {
                g.w[t] = t < nt ? a.w[scalar + (t0 + t) * a.H] : 0.f;
                g.beta[t] = t < nt ? a.beta[scalar + (t0 + t) * a.H] : 0.f;
            }
            cp_async_commit();
            cp_async_wait();
            bar_sync<G::STAGERS>(kBarStage);
            split_rows<BLK, N, G::LDR, LD, KE, G::STAGERS>(g.e, G::PIECE, g.raw, stid);
            split_rows<BLK, N, G::LDR, LD, KD, G::STAGERS>(g.du, G::PIECE, g.raw + G::ROW, stid);
            if constexpr (KP == 3) split_rows<BLK, N, G::LDR, LD, 3, G::STAGERS>(g.dy, G::PIECE, g.raw + 2 * G::ROW, stid);
            if constexpr (!GRAD) {
                if (slice == 0) {   // dbeta: du . e, eight lanes a token
#pragma unroll
                    for (int t = stid / 8; t < BLK; t += G::STAGERS / 8) {
                        float x = 0.f;
#pragma unroll
                        for (int j = lane % 8; j < N; j += 8) x = fmaf(g.raw[t * G::LDR + j], g.raw[G::ROW + t * G::LDR + j], x);
                        x += __shfl_xor_sync(0xffffffffu, x, 1);
                        x += __shfl_xor_sync(0xffffffffu, x, 2);
                        x += __shfl_xor_sync(0xffffffffu, x, 4);
                        if (lane % 8 == 0 && t < nt) a.dbeta[scalar + (t0 + t) * a.H] = x;
                    }
                }
            }
            bar_sync<G::STAGERS>(kBarStage);
            // the two matrices of each chunk, one a warp at a time
            float* gam = reinterpret_cast<float*>(smem + 2 * G::STAGE + G::B_RAW) + (warp - NW) * G::SCR;
            for (int j = warp - NW; j / 2 * kChunk < nt; j += G::STAGERS / 32) {
                const int c = j / 2, which = j % 2;
                const float* be = g.beta + c * kChunk;
                const ChunkDecay d = chunk_decay(g.w + c * kChunk, gam, lane);
                if (which == 0 && lane < 16) {
                    g.sc[c * kChunk + tl] = d.upto;
                    g.sc[BLK + c * kChunk + tl] = d.upto * be[tl];
                    g.sc[2 * BLK + c * kChunk + tl] = d.after * be[tl];
                }
                __syncwarp();
                const __nv_bfloat16 *ec = g.e + c * kChunk * LD, *dc = g.du + c * kChunk * LD, *yc = g.dy + c * kChunk * LD;
                __nv_bfloat16* m = g.mats + (c * (G::M0 + G::M1) + (which ? G::M0 : 0)) * G::MAT;
                float x[2][4];
                if constexpr (!GRAD) {
                    // 0: G[t][s] beta_s beta_t e_s.du_t (s < t); 1: G[t][s] beta_s e_s.dy_t (s <= t)
                    if (which == 0) gram<N, KD, KE, PP>(x, dc, ec, G::PIECE, lane);
                    else gram<N, KP, KE, 3>(x, yc, ec, G::PIECE, lane);
                } else {
                    // 0: G[s][t] beta_t e_t.dy_s (s >= t); 1: -G[s][t] beta_s beta_t e_t.du_s (s > t)
                    if (which == 0) gram<N, KE, KP, PP>(x, ec, yc, G::PIECE, lane);
                    else gram<N, KE, PP, PP>(x, ec, dc, G::PIECE, lane);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int hrow = 0; hrow < 2; ++hrow) {
                        const int t = lane / 4 + 8 * hrow, s0 = 8 * n + 2 * (lane % 4);
                        float v[2];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int s = s0 + q;
                            const float gm = GRAD ? gam[s * 17 + t] : gam[t * 17 + s];
                            float f;
                            if constexpr (!GRAD) f = which == 0 ? (s < t ? gm * be[s] * be[t] : 0.f) : gm * be[s];
                            else f = which == 0 ? gm * be[t] : (s > t ? -gm * be[s] * be[t] : 0.f);
                            v[q] = f * x[n][2 * hrow + q];
                        }
                        if (which == 0) put_pieces<G::M0>(m, t, s0, v[0], v[1]);
                        else put_pieces<G::M1>(m, t, s0, v[0], v[1]);
                    }
                __syncwarp();
            }
            bar_arrive<G::THREADS>(kBarFull + st);
        }
        return;
    }

    const int i0 = warp * 16;
    const int64_t nchunk = (a.T + kCheck - 1) / kCheck;
    const int slot = slice / 16 + warp;
    float* ck = a.check + head * (nchunk + 1) * N * N + slot * (N * 16);
    float* phi = a.phi + head * (nchunk + 1) * G::SLOTS + slot;
    float* pr = a.pr + slot * (a.B * a.T * a.H) + scalar;
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

    const bool own = a.H == a.Hk;
    const int off_b = b_plain(lane, LD), off_t = b_trans(lane, LD), off_m = b_plain(lane, kMatLd);
    int st = 0;
    int64_t t0 = first;
    for (int64_t i = 0; i < blocks; ++i, t0 += step, st ^= 1) {
        const int nt = a.T - t0 < BLK ? int(a.T - t0) : BLK;
        const int nch = (nt + kChunk - 1) / kChunk;
        G g(smem, st);
        if (!GRAD && t0 % kCheck == 0) keep(t0 / kCheck);
        bar_sync<G::THREADS>(kBarFull + st);
#pragma unroll 1
        for (int cc = 0; cc < nch; ++cc) {
            const int c = GRAD ? nch - 1 - cc : cc;
            const __nv_bfloat16 *ec = g.e + c * kChunk * LD, *dc = g.du + c * kChunk * LD, *yc = g.dy + c * kChunk * LD;
            const __nv_bfloat16* m0 = g.mats + c * (G::M0 + G::M1) * G::MAT;
            const __nv_bfloat16* m1 = m0 + G::M0 * G::MAT;
            const float* sc = g.sc + c * kChunk;
            IO *kt = g.k + c * kChunk * G::LDV + i0, *rt = g.r + c * kChunk * G::LDV + i0;
            const int64_t t = t0 + c * kChunk, at = base + t * vs + slice + i0;
            const int left = nt - c * kChunk;
            float k[2][4], r[2][4];
            load_lines(k, kt, G::LDV, lane);
            load_lines(r, rt, G::LDV, lane);
            uint32_t kq[KP][4];
            split_a<KP>(k[0], k[1], kq);
            const float gl = sc[kChunk - 1];
            if constexpr (!GRAD) {
                float o1[2][4], o2[2][4];
                {
                    Acc pa, qa;
#pragma unroll
                    for (int kk = 0; kk < N / 16; ++kk) {
                        uint32_t sp[3][4];
                        split_a<3>(S[2 * kk], S[2 * kk + 1], sp);
                        times<3, KD, PP, false>(pa, kk == 0, sp, dc + kk * 16, G::PIECE, off_b);
                        times<3, KP, 3, false>(qa, kk == 0, sp, yc + kk * 16, G::PIECE, off_b);
                    }
                    pa.sum(o1);
                    qa.sum(o2);
                    scale_tokens(o1, sc + BLK, lane);
                    scale_tokens(o2, sc, lane);
                }
                {
                    Acc pa, qa;
                    times<KP, G::M0, PP, false>(pa, true, kq, m0, G::MAT, off_m);
                    times<KP, G::M1, 3, false>(qa, true, kq, m1, G::MAT, off_m);
                    float p[2][4], q[2][4];
                    pa.sum(p);
                    qa.sum(q);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o1[n][x] = -(o1[n][x] + p[n][x]), o2[n][x] += q[n][x];
                }
                // S <- g_15 S + (G beta k) e^T
                scale_tokens(k, sc + 2 * BLK, lane);
                uint32_t k3[3][4];
                split_a<3>(k[0], k[1], k3);
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    float d[2][4];
                    times_add<3, 3>(d, true, k3, ec + kk * 16, G::PIECE, off_t);
                    fade_add(S[2 * kk], gl, d[0]);
                    fade_add(S[2 * kk + 1], gl, d[1]);
                }
                store_lines(a.dkh + at, vs, left, o1, kt, 0, false, lane);
                token_sums(pr + t * a.H, a.H, left, o2, r, lane);
                if (own) store_lines(static_cast<IO*>(a.dr) + at, vs, left, o2, rt, G::LDV, a.vec, lane);
                else store_lines(a.drh + at, vs, left, o2, rt, 0, false, lane);
            } else {
                // the state's part of dk, on its way while the rest is formed
                float o0[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int tt = 8 * n + 2 * (lane % 4) + (x & 1);
                        o0[n][x] = tt < left ? __ldcg(a.dkh + at + tt * vs + lane / 4 + (x >> 1) * 8) : 0.f;
                    }
                uint32_t rq[KP][4];
                split_a<KP>(r[0], r[1], rq);
                float o[2][4];
                {
                    Acc pa;
#pragma unroll
                    for (int kk = 0; kk < N / 16; ++kk) {
                        uint32_t sp[PP][4];
                        split_a<PP>(S[2 * kk], S[2 * kk + 1], sp);
                        times<PP, KE, PP, false>(pa, kk == 0, sp, ec + kk * 16, G::PIECE, off_b);
                    }
                    pa.sum(o);
                    scale_tokens(o, sc + 2 * BLK, lane);
                }
                {
                    Acc pa;
                    times<KP, G::M0, PP, false>(pa, true, rq, m0, G::MAT, off_m);
                    times<KP, G::M1, PP, false>(pa, false, kq, m1, G::MAT, off_m);
                    float p[2][4];
                    pa.sum(p);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[n][x] += p[n][x], k[n][x] = -k[n][x];
                }
                // D <- g_15 D + (g r) dy^T - (g beta k) du^T
                scale_tokens(r, sc, lane);
                scale_tokens(k, sc + BLK, lane);
                uint32_t r3[3][4], k3[3][4];
                split_a<3>(r[0], r[1], r3);
                split_a<3>(k[0], k[1], k3);
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    float d[2][4];
                    times_add<3, 3>(d, true, k3, dc + kk * 16, G::PIECE, off_t);
                    times_add<3, KP>(d, false, r3, yc + kk * 16, G::PIECE, off_t);
                    fade_add(S[2 * kk], gl, d[0]);
                    fade_add(S[2 * kk + 1], gl, d[1]);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[n][x] += o0[n][x];
                if (own) store_lines(static_cast<IO*>(a.dk) + at, vs, left, o, kt, G::LDV, a.vec, lane);
                else store_lines(a.dkh + at, vs, left, o, kt, 0, false, lane);
            }
        }
        if (GRAD && t0 % kCheck == 0) border(t0 / kCheck);
        if (i + 2 < blocks) bar_arrive<G::THREADS>(kBarFree + st);
    }
    if constexpr (!GRAD) keep(nchunk);
}

// dr and dk of a key head: the sums over the value heads that share it, in
// their order.  One thread per 4 channels.
template <typename IO, int N>
__global__ void __launch_bounds__(256) delta_share_kernel(const Args a) {
    const int64_t id = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (id >= a.B * a.T * a.Hk * (N / 4)) return;
    const int64_t key = id / (N / 4);   // (sequence, token, key head)
    const int share = int(a.H / a.Hk), c = int(id % (N / 4)) * 4;
    const float* pr = a.drh + key * share * N + c;
    const float* pk = a.dkh + key * share * N + c;
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f), k = r;
    for (int s = 0; s < share; ++s) {
        const float4 x = *reinterpret_cast<const float4*>(pr + s * N), y = *reinterpret_cast<const float4*>(pk + s * N);
        r.x += x.x, r.y += x.y, r.z += x.z, r.w += x.w;
        k.x += y.x, k.y += y.y, k.z += y.z, k.w += y.w;
    }
    IO* orr = static_cast<IO*>(a.dr) + key * N + c;
    IO* ok = static_cast<IO*>(a.dk) + key * N + c;
    put(orr, r.x), put(orr + 1, r.y), put(orr + 2, r.z), put(orr + 3, r.w);
    put(ok, k.x), put(ok + 1, k.y), put(ok + 2, k.z), put(ok + 3, k.w);
}

// dw of a chunk of kCheck tokens: the sum <Dn, S> from the chunk's end
// backwards; its first token's is the border's own.  One thread per
// (sequence, chunk, head).
template <int SLOTS>
__global__ void __launch_bounds__(64) delta_dw_kernel(const Args a) {
    const int64_t nchunk = (a.T + kCheck - 1) / kCheck;
    const int64_t id = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (id >= a.B * nchunk * a.H) return;
    const int64_t h = id % a.H, c = id / a.H % nchunk, b = id / a.H / nchunk;
    const float* phi = a.phi + ((b * a.H + h) * (nchunk + 1) + c) * SLOTS;
    float first = 0.f, x = 0.f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) first += phi[s], x += phi[SLOTS + s];
    const int64_t t0 = c * kCheck, t1 = t0 + kCheck < a.T ? t0 + kCheck : a.T;
    const int64_t plane = a.B * a.T * a.H;
    constexpr int U = 8;   // tokens whose loads are in flight at once
    for (int64_t t = t1 - 1; t > t0; t -= U) {
        float term[U], w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = (b * a.T + (t - u > t0 ? t - u : t0)) * a.H + h;
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < SLOTS; ++q) s += a.pr[q * plane + at] - a.pv[q * plane + at];
            term[u] = s;
            w[u] = a.w[at];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x += term[u];
            // a state that nothing is left of has no gradient, whatever the sum's rounding left
            if (t - u > t0) a.dw[(b * a.T + t - u) * a.H + h] = expf(-w[u]) == 0.f ? 0.f : -x;
        }
    }
    a.dw[(b * a.T + t0) * a.H + h] = -first;
}

}  // namespace delta
}  // namespace wkv
