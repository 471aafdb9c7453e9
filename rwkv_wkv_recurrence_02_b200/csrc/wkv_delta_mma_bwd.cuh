// wkv_delta_mma_bwd.cuh -- reverse mode of the gated delta rule on the tensor
// cores (wkv_delta_mma.cuh has the notation, the layouts and how float32
// accuracy is kept).
//
// Within a chunk left by gradient state D (of the state after it), G[t][s]
// the decays of tokens s+1 .. t, g_t those up to t, q_t those after t:
//   (I + B)^T DU = diag(q) D^T K + P^T DY,   B[s][t] = G[s][t] beta_s k_s.k_t  (t < s)
//                                            P[s][t] = G[s][t] r_s.k_t         (t <= s)
//   dv = beta du
//   D  <- g_15 D + R^T diag(g) DY - K^T diag(g beta) DU
// with the state S that enters and u = beta e:
//   dr_t = g_t S dy_t + sum_{s<=t} G[t][s] (u_s.dy_t) k_s
//   dk_t = q_t D u_t + sum_{s>=t} G[s][t] (dy_s.u_t) r_s - sum_{s>t} G[s][t] (dv_s.u_t) k_s
//          - g_t S dv_t - sum_{s<t} G[t][s] (u_s.dv_t) k_s
// Two walks, for e and the states between segments of 64 tokens (the forward
// kernel) and for du and the gradient states between them; with those, dr and
// dk of a segment need nothing from the others, and a third kernel forms them
// for every segment at once.  It starts dw from the inner product <D, S> at the
// segment's end.  The two walks run side by side in one kernel.
//
// Measured, bfloat16: 8 x 4096 tokens of 32 heads of 64 1735 us (reads and writes
// alone: 150), the walks 870 of it, bound as the forward is, the segments
// the rest (wkv_delta_tc.cuh).  2047 tokens of 16 heads of 128, 8 key heads: 343 us,
// 220 of it the walks (64 CTAs, a chunk's chain), 120 the segments: one CTA an SM, the
// tensor pipe active in 35% of the cycles, first among its stalls.
// The two walks one after the other took 671 us on 4096 tokens of 32 heads of
// 64 where side by side all kernels took 414 (406 now).
#pragma once

#include "wkv_delta_mma.cuh"

namespace wkv {
namespace delta {

// ---------------------------------------------------------------------------
// du, dv, the initial state's gradient and the gradient states between
// segments (value columns, backwards)
// ---------------------------------------------------------------------------
template <typename IO, int N>
using ReverseShape = Columns<IO, N, true, 6, 3>;

// A chunk's nt tokens of a warp's 16 columns one after another, backwards, from the
// staged rows (S: D^T); du and dv at the lane's first line.  w, beta: of its first token.
template <typename IO, int N>
__device__ __forceinline__ void reverse_tokens(const ReverseShape<IO, N>& g, float (&S)[N / 8][4], int j0, int nt, const float* w,
                                               const float* beta, int64_t heads, float* du, IO* dv, int64_t vs, int lane) {
    using G = ReverseShape<IO, N>;
#pragma unroll 1
    for (int t = nt - 1; t >= 0; --t) {
        const __nv_bfloat16* kp = g.k + t * G::LD + 2 * (lane % 4);
        const IO* yp = g.v + t * G::LDV + j0 + lane / 4;
        const float a = expf(-w[t * heads]), be = beta[t * heads], dy[2] = {to_f32(yp[0]), to_f32(yp[8])};
        float x[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < N / 8; ++n) {
            const float2 k = staged_pair<G::KP>(kp + 8 * n, G::PIECE), r = staged_pair<G::KP>(kp + (g.r() - g.k) + 8 * n, G::PIECE);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                S[n][i] = fmaf((i & 1) ? r.y : r.x, dy[i >> 1], S[n][i]);
                x[i >> 1] = fmaf(S[n][i], (i & 1) ? k.y : k.x, x[i >> 1]);
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            x[q] = quad_sum(x[q]);
            if (lane % 4 == 0) du[t * vs + 8 * q] = x[q];
            x[q] *= be;
            if (lane % 4 == 0) put(dv + t * vs + 8 * q, x[q]);
        }
#pragma unroll
        for (int n = 0; n < N / 8; ++n) {
            const float2 k = staged_pair<G::KP>(kp + 8 * n, G::PIECE);
#pragma unroll
            for (int i = 0; i < 4; ++i) S[n][i] = a * fmaf((i & 1) ? k.y : k.x, -x[i >> 1], S[n][i]);
        }
    }
}

// where the gradient of the state ahead of the walk's first token goes
template <int N, bool PARTS, typename PLACE>
__device__ __forceinline__ void reverse_end(const Args& a, const PLACE& p, const float (&S)[N / 8][4], int lane) {
    if (PARTS && p.begin > 0) hand_on<N>(p.hand(a), S, lane);
    else if (a.ds_in != nullptr) store_state<N>(a.ds_in + p.head * N * N + p.column, S, lane);
}
template <typename IO, int N, bool PARTS>
__device__ __noinline__ void reverse_again(const Args& a, char* smem, const Task& task) {
    using G = ReverseShape<IO, N>;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t nseg = (a.T + kSegment - 1) / kSegment, vs = a.H * N;
    const Reach<G, N, PARTS, true> p(a, task, warp);
    float S[N / 8][4];
    p.start(S, a, task, a.ds_out, lane);
    int st = 0;
#pragma unroll 1
    for (int64_t t0 = p.begin + (p.end - 1 - p.begin) / kChunk * kChunk; t0 >= p.begin; t0 -= kChunk, st = (st + 1) % G::NST) {
        const int nt = p.end - t0 < kChunk ? int(p.end - t0) : kChunk;
        const int64_t row = p.row + t0 * a.H, line = p.values + t0 * vs + lane / 4;
        bar_sync<G::BAR>(kBarFull + st);
        reverse_tokens<IO, N>(G(smem, st), S, warp * 16, nt, a.w + row, a.beta + row, a.H, a.du + line, static_cast<IO*>(a.dv) + line, vs, lane);
        if (t0 >= p.begin + G::NST * kChunk) bar_arrive<G::BAR>(kBarFree + st);
        if (t0 % kSegment == 0) keep_state<IO, N>(a.d_seg + (p.head * (nseg + 1) + t0 / kSegment) * N * N, p.column, S, lane);
    }
    reverse_end<N, PARTS>(a, p, S, lane);
}

template <typename IO, int N, bool PARTS>
__device__ __forceinline__ void reverse_walk(const Args& a, char* smem, int64_t block) {
    using G = ReverseShape<IO, N>;
    constexpr int KP = G::KP, LD = G::LD;
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
            const int64_t begin = PARTS ? (a.parts - 1 - task.part) * a.part_len : 0;
            const int64_t end = PARTS && begin + a.part_len < a.T ? begin + a.part_len : a.T;
            const int64_t last = begin + (end - 1 - begin) / kChunk * kChunk;
            const int64_t vbase = (b * a.T * a.H + h) * N + task.walk % G::SLICES * G::CW;
            const IO* kp = static_cast<const IO*>(a.k) + (b * a.T * a.Hk + hk) * N;
            const IO* rp = static_cast<const IO*>(a.r) + (b * a.T * a.Hk + hk) * N;
            const IO* yp = static_cast<const IO*>(a.dy) + vbase;
            const float* wp = a.w + b * a.T * a.H + h;
            const float* bp = a.beta + b * a.T * a.H + h;
            bool again = false;
            do {
#pragma unroll 1
                for (int64_t t0 = last - st * kChunk; t0 >= begin; t0 -= G::NST * kChunk) {
                    const int nt = end - t0 < kChunk ? int(end - t0) : kChunk;
                    if (last - t0 >= G::NST * kChunk) bar_sync<G::BAR>(kBarFree + st);
                    const float w = lane < nt ? wp[(t0 + lane) * a.H] : 0.f, be = lane < nt ? bp[(t0 + lane) * a.H] : 0.f;
                    g.fetch(kp + t0 * ks, rp + t0 * ks, ks, yp + t0 * vs, vs, nt, a.vec, lane);
                    // B, its inverse and P
                    const ChunkDecay d = chunk_decay<kChunk>(w, g.sums, lane);
                    if (lane < kChunk) {
                        g.beta[lane] = be;
                        g.sc[lane] = d.after;
                        g.sc[kChunk + lane] = d.upto;
                        g.sc[2 * kChunk + lane] = d.upto * be;
                    }
                    __syncwarp();
                    float kk[2][4], rk[2][4];
                    gram<N, KP, KP, KP, kChain<IO>>(kk, g.k, g.k, G::PIECE, lane);
                    gram<N, KP, KP, KP, kChain<IO>>(rk, g.r(), g.k, G::PIECE, lane);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int t = 8 * n + 2 * (lane % 4);
                        const float2 t0s = g.sums[t], t1s = g.sums[t + 1];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int s = lane / 4 + 8 * q;
                            const float bs = g.beta[s];
                            const float2 ss = g.sums[s];
                            const float g0 = decay_of(ss, t0s), g1 = decay_of(ss, t1s);
                            g.diag[s * 20 + t] = t < s ? g0 * bs * kk[n][2 * q] : 0.f;
                            g.diag[s * 20 + t + 1] = t + 1 < s ? g1 * bs * kk[n][2 * q + 1] : 0.f;
                            put_pieces<3>(g.mats + 3 * kMat, s, t, t <= s ? g0 * rk[n][2 * q] : 0.f,
                                          t + 1 <= s ? g1 * rk[n][2 * q + 1] : 0.f);
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
    const int off_b = b_plain(lane, LD), off_t = b_trans(lane, LD), off_m = m_trans(lane);
    using Place = Reach<G, N, PARTS, true>;
    for (; next_task<PARTS, G::THREADS>(a, walks, block, task, first); first = false) {
        const Place here(a, task, warp);
        const int64_t begin = here.begin, end = here.end;
        const int64_t last = begin + (end - 1 - begin) / kChunk * kChunk;
        float* grads = a.d_seg + here.head * (nseg + 1) * N * N;
        float S[N / 8][4];   // D^T
        here.start(S, a, task, a.ds_out, lane);
        // gradient states between segments, as S^T's
        if (!PARTS || task.part == 0) keep_state<IO, N>(grads + nseg * N * N, here.column, S, lane);
        int st = 0;
#pragma unroll 1
        for (int64_t t0 = last; t0 >= begin; t0 -= kChunk, st = (st + 1) % G::NST) {
            const int nt = end - t0 < kChunk ? int(end - t0) : kChunk;
            G g(smem, st);
            bar_sync<G::BAR>(kBarFull + st);
            // X = diag(q) D^T K + P^T dY
            float dy[2][4], x[2][4];
            {
                Acc pa;
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    uint32_t sp[3][4];
                    split_a<3>(S[2 * kk], S[2 * kk + 1], sp);
                    times<3, KP, 3, false>(pa, pa.template start<kChain<IO>>(x, kk), kk == 0, sp, g.k + kk * 16, G::PIECE, off_b);
                }
                pa.template finish<kChain<IO>>(x, N / 16);
            }
            load_lines(dy, g.v + j0, G::LDV, lane);
            scale_tokens(x, g.sc, lane);
            {
                uint32_t yq[KP][4];
                split_a<KP>(dy[0], dy[1], yq);
                Acc ya;
                times<KP, 3, 3, true>(ya, true, true, yq, g.mats + 3 * kMat, kMat, off_m);
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
                times<3, 3, 3, true>(ea, true, true, xp, g.mats, kMat, off_m);
                ea.sum(du);
            }
            // D <- g_15 D + (g dy)^T R - (g beta du)^T K
            {
                float f1[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) f1[n][i] = -du[n][i];
                scale_tokens(dy, g.sc + kChunk, lane);
                scale_tokens(f1, g.sc + 2 * kChunk, lane);
                uint32_t yq[3][4], uq[3][4];
                split_a<3>(dy[0], dy[1], yq);
                split_a<3>(f1[0], f1[1], uq);
                const float gl = g.sc[2 * kChunk - 1];
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) {
                    float d[2][4];
                    times_add<3, KP>(d, true, uq, g.k + kk * 16, G::PIECE, off_t);
                    times_add<3, KP>(d, false, yq, g.r() + kk * 16, G::PIECE, off_t);
                    fade_add(S[2 * kk], gl, d[0]);
                    fade_add(S[2 * kk + 1], gl, d[1]);
                }
            }
            const int64_t at = here.values + t0 * vs;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                store_half(a.du + at + 8 * n * vs, vs, nt - 8 * n, du[n], g.v, 0, false, lane);
                const float2 be = pair_at(g.beta, n, lane);
#pragma unroll
                for (int i = 0; i < 4; ++i) du[n][i] *= (i & 1) ? be.y : be.x;
                // dv through dy's columns, which only this warp reads
                store_half(static_cast<IO*>(a.dv) + at + 8 * n * vs, vs, nt - 8 * n, du[n], g.v + 8 * n * G::LDV + j0, G::LDV, a.vec, lane);
            }
            if (t0 >= begin + G::NST * kChunk) bar_arrive<G::BAR>(kBarFree + st);
            if (t0 % kSegment == 0) keep_state<IO, N>(grads + t0 / kSegment * N * N, here.column, S, lane);
        }
        const uint32_t odd = odd_lines<N>(S);
        if (bar_or<G::THREADS>(kBarTask, odd != 0 && began_finite<N, Place>(a, task, a.ds_out, odd))) {   // as in the forward walk
            reverse_again<IO, N, PARTS>(a, smem, task);
            continue;
        }
        reverse_end<N, PARTS>(a, here, S, lane);
    }
}

template <typename IO, int N>
__global__ void __launch_bounds__(ReverseShape<IO, N>::THREADS, kCtas<IO, N>) delta_reverse_mma_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(16) char smem[];
    pdl_wait();
    reverse_walk<IO, N, true>(a, smem, blockIdx.x);
}
// Whole walks of both kinds: they need nothing of each other.  The reverse
// ones, which take longer, first: 4 x 4096 tokens of 24 heads of 64 737 us, 815 the
// other way round (8 x 4096 of 32 heads 1741 and 1727).  In turn they take 938 and
// 2032 us, and 481 where 32 heads of one sequence take 406: both codes in one
// instruction cache.
template <typename IO, int N>
__global__ void __launch_bounds__(ReverseShape<IO, N>::THREADS, kCtas<IO, N>) delta_walks_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(16) char smem[];
    const int64_t walks = a.B * a.H * ReverseShape<IO, N>::SLICES;
    pdl_wait();
    if (blockIdx.x < walks) reverse_walk<IO, N, false>(a, smem, blockIdx.x);
    else forward_walk<IO, N, false, false>(a, smem, blockIdx.x - walks);
}

// ---------------------------------------------------------------------------
// dr, dk, dbeta and dw of one segment.  A warp takes 16 tokens t and IC
// channels i: the products with S and D, then those with K and R of the
// segment's 16 x 16 blocks of (token, token) products.  A block is formed once,
// by one warp, and read from shared memory as it lies and transposed.
// ---------------------------------------------------------------------------
// 16 x 32 of a warp's: 343 us for 2047 tokens of 16 heads of 128 (the whole call), as
// with 16 x 64, whose warps are half as many (segment_tokens wants four threads a
// key).  Bfloat16 heads of 64 take wkv_delta_tc.cuh's kernel.
template <typename IO, int N>
struct SegmentShape {
    static constexpr int KP = sizeof(IO) == 2 ? 1 : 3;
    static constexpr int IC = 32, PARTS = N / IC;
    static constexpr int WARPS = 4 * PARTS, THREADS = 32 * WARPS;
    static constexpr int PIECE = kSegment * N;                // rows without padding (Swizzled)
    static constexpr int JB = 32;                             // value lines of S and D at a time
    static constexpr int SPIECE = JB * N;
    static constexpr int BLOCKS = 10, MATS = 6;               // blocks of token pairs on and below the diagonal, pieces of each
    // u, dv, dy; S and D, later the blocks; K and R (float32's over the rows when
    // those are done with); the decays and the sums over channels
    static constexpr int S_ROWS = (6 + KP) * PIECE * 2;
    static constexpr int A_ = 6 * SPIECE * 2, B_ = BLOCKS * MATS * kMat * 2, S_BUF = A_ > B_ ? A_ : B_;
    static constexpr int S_KEYS = KP == 1 ? 2 * PIECE * 2 : 0;
    static constexpr int S_SUM = kSegment * (8 + 4 + 4 * PARTS) + WARPS * 8;
    static constexpr int SMEM = S_ROWS + S_BUF + S_KEYS + S_SUM;
    // CTAs an SM by shared memory; registers follow
    static constexpr int CTAS = 227 * 1024 / (SMEM + 1024) > 3 ? 3 : 227 * 1024 / (SMEM + 1024);
};

// d[p] += f (A B), f0 and f1 the factors of the lane's two rows: A 16 tokens and
// 32 columns (NA pieces from a_at on, `ap` bytes apart; col: the lane's place in
// them), B 32 lines (NB pieces from b_at on, `bp` apart; ch: its place in channels)
template <int N, int NA, int NB, int ORD, int NP>
__device__ __forceinline__ void add_lines(float (&d)[NP][2][4], float f0, float f1, uint32_t a_at, int ap, uint32_t col,
                                          uint32_t b_at, int bp, uint32_t ch) {
    uint32_t a[2][NA][4];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int c = 0; c < NA; ++c) ldsm4(a[kk][c], a_at + (col ^ (kk * 32)) + c * ap);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        float x[2][4];
        bool first = true;
        uint32_t b[2][NB][4];
#pragma unroll
        for (int c = NB - 1; c >= 0; --c)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) ldsm4t(b[kk][c], b_at + (ch ^ (p * 32)) + kk * (16 * N * 2) + c * bp);
#pragma unroll
        for (int o = ORD - 1; o >= 0; --o)   // smallest orders first
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int c = 0; c < NA && c <= o; ++c)
                    if (o - c < NB) {
                        mma2(x, a[kk][c], b[kk][o - c], first);
                        first = false;
                    }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            fma_pair(d[p][n][0], d[p][n][1], f0, x[n][0], x[n][1]);
            fma_pair(d[p][n][2], d[p][n][3], f1, x[n][2], x[n][3]);
        }
    }
}

// what a CTA of the segments' kernels works on
struct Segment {
    int64_t head, seg, ks, vs;   // strides of a token in keys and values
    int64_t state;               // of its first state among those between segments
    int64_t rows, keys, scalar;  // of its first token in values, keys and per-head scalars
    int nt;                      // tokens
    __device__ __forceinline__ Segment(const Args& a, int N, int64_t block) {
        // heads first: neighbours in memory are worked on at the same time.  All of
        // these fit 32 bits, as the grid does.
        const uint32_t H = uint32_t(a.H), nseg = uint32_t((a.T + kSegment - 1) / kSegment), id = uint32_t(block);
        const uint32_t q = id / H, h = id - q * H, hk = h / (H / uint32_t(a.Hk)), b32 = q / nseg;
        seg = q - b32 * nseg;
        const int64_t b = b32, t0 = seg * kSegment;
        head = b * a.H + h;
        nt = a.T - t0 < kSegment ? int(a.T - t0) : kSegment;
        ks = a.Hk * N, vs = a.H * N;
        state = (head * (nseg + 1) + seg) * N * N;
        rows = ((b * a.T + t0) * a.H + h) * N, keys = ((b * a.T + t0) * a.Hk + hk) * N;
        scalar = (b * a.T + t0) * a.H + h;
    }
};

// A warp's RW rows of u = beta e and dv = beta du (three pieces each), at their
// places in shared memory; dbeta, and dv . v of a token.
template <typename IO, int N, int RW, typename AT>
__device__ __forceinline__ void stage_values(const Args& a, const Segment& sg, __nv_bfloat16* ub, __nv_bfloat16* db, int piece, AT place,
                                             int row, float* dvv, int lane) {
    constexpr int KP = sizeof(IO) == 2 ? 1 : 3;
    const int left = sg.nt - row;
    const int64_t rows = sg.rows, vs = sg.vs, scalar = sg.scalar;
    constexpr int ROWV = N / 4, ALL = RW * ROWV / 32, U = ALL < 8 ? ALL : 8;
#pragma unroll 1
    for (int n = 0; n < ALL; n += U) {
        // all loads first, of a row that exists; rows behind the last token are zeroed after
        float4 x[U], y[U], v[U];
        uint2 vr[U];
        float be[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = lane + (n + u) * 32, t = i / ROWV, c = (i % ROWV) * 4;
            const int64_t at = rows + (t < left ? row + t : 0) * vs + c;
            be[u] = __ldg(a.beta + scalar + (t < left ? row + t : 0) * a.H);
            x[u] = load4(a.e + at, true);
            y[u] = load4(a.du + at, true);
            const IO* vp = static_cast<const IO*>(a.v) + at;
            if constexpr (KP == 3) {
                v[u] = load4(reinterpret_cast<const float*>(vp), a.vec);
            } else if (a.vec) {
                vr[u] = __ldg(reinterpret_cast<const uint2*>(vp));
            } else {
                const unsigned short* q = reinterpret_cast<const unsigned short*>(vp);
                vr[u] = make_uint2(q[0] | uint32_t(q[1]) << 16, q[2] | uint32_t(q[3]) << 16);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = lane + (n + u) * 32, t = i / ROWV, c = (i % ROWV) * 4;
            if constexpr (KP == 1)
                v[u] = make_float4(__uint_as_float(vr[u].x << 16), __uint_as_float(vr[u].x & 0xffff0000u),
                                   __uint_as_float(vr[u].y << 16), __uint_as_float(vr[u].y & 0xffff0000u));
            if (t >= left) x[u] = y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            const float bt = be[u];
            float s = fmaf(x[u].x, y[u].x, fmaf(x[u].y, y[u].y, fmaf(x[u].z, y[u].z, x[u].w * y[u].w)));
            float z = fmaf(v[u].x, y[u].x, fmaf(v[u].y, y[u].y, fmaf(v[u].z, y[u].z, v[u].w * y[u].w)));
#pragma unroll
            for (int o = ROWV / 2; o > 0; o /= 2) {
                s += __shfl_xor_sync(0xffffffffu, s, o);
                z += __shfl_xor_sync(0xffffffffu, z, o);
            }
            if (lane % ROWV == 0) {
                if (t < left) a.dbeta[scalar + (row + t) * a.H] = s;
                dvv[row + t] = bt * z;
            }
            put4<3>(ub + place(row + t, c), piece, make_float4(bt * x[u].x, bt * x[u].y, bt * x[u].z, bt * x[u].w));
            put4<3>(db + place(row + t, c), piece, make_float4(bt * y[u].x, bt * y[u].y, bt * y[u].z, bt * y[u].w));
        }
    }
}

// the decays' running sum, two tokens a lane (one warp); returns their rates
__device__ __forceinline__ float2 segment_sums(const Args& a, const Segment& sg, float2* sums, int lane) {
    const int64_t scalar = sg.scalar;
    const int nt = sg.nt;
    const int ta = 2 * lane;
    const float w0 = ta < nt ? a.w[scalar + ta * a.H] : 0.f, w1 = ta + 1 < nt ? a.w[scalar + (ta + 1) * a.H] : 0.f;
    const double x0 = w0 > kMaxRate ? kMaxRate : w0, x1 = x0 + double(w1 > kMaxRate ? kMaxRate : w1);
    double x = x1;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    sums[ta] = two_floats(x - x1 + x0);
    sums[ta + 1] = two_floats(x);
    return make_float2(w0, w1);
}

// own: r . dr of the lane's two rows over its warp's channels (R's pieces staged)
template <int N, int NP, int KP>
__device__ __forceinline__ void row_products(float (&own)[2], const __nv_bfloat16* rb, int piece, const float (&dr)[NP][2][4], int t_lo,
                                             int i0, int lane) {
    constexpr Swizzled<N> place{};
    own[0] = own[1] = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const __nv_bfloat16* r2 = rb + place(t_lo + 8 * q, i0 + p * 16 + 8 * n + 2 * (lane % 4));
                const float2 x = staged_pair<KP>(r2, piece);
                own[q] = fmaf(x.x, dr[p][n][2 * q], fmaf(x.y, dr[p][n][2 * q + 1], own[q]));
            }
}

// dr and dk of a warp's 16 tokens and its channels; tile: shared memory of the
// warp's own for bfloat16's 16-byte stores
template <typename IO, int N, int NP>
__device__ __forceinline__ void store_rows(const Args& a, const Segment& sg, const float (&dr)[NP][2][4], const float (&dk)[NP][2][4],
                                           __nv_bfloat16* tile, int tb, int i0, int lane) {
    constexpr int KP = sizeof(IO) == 2 ? 1 : 3;
    const int64_t rows = sg.rows, vs = sg.vs;
    const int nt = sg.nt, t_lo = tb * 16 + lane / 4;
    const bool whole = a.H == a.Hk;
    if (!whole || KP == 3) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int t = t_lo + 8 * q;
            if (t >= nt) continue;
            const int64_t at = rows + t * vs + i0 + 2 * (lane % 4);
            float* orr = (whole ? static_cast<float*>(a.dr) : a.drh) + at;
            float* ok = (whole ? static_cast<float*>(a.dk) : a.dkh) + at;
            const bool pairs = !whole || a.vec;
#pragma unroll
            for (int c = 0; c < 2 * NP; ++c) {
                const float *x = &dr[c / 2][c % 2][2 * q], *y = &dk[c / 2][c % 2][2 * q];
                if (pairs) {
                    *reinterpret_cast<float2*>(orr + 8 * c) = make_float2(x[0], x[1]);
                    *reinterpret_cast<float2*>(ok + 8 * c) = make_float2(y[0], y[1]);
                } else {
                    orr[8 * c] = x[0], orr[8 * c + 1] = x[1];
                    ok[8 * c] = y[0], ok[8 * c + 1] = y[1];
                }
            }
        }
    } else if constexpr (KP == 1) {   // through rows of the warp's own (where u was) to 16-byte stores
        constexpr int LD = 16 * NP + 8;
        const uint32_t to = smem_u32(tile + ((lane & 7) + ((lane >> 3) & 1) * 8) * LD + (lane >> 4) * 8);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            stsm_tile(to + p * 32, dr[p]);
            stsm_tile(to + (16 * LD + p * 16) * 2, dk[p]);
        }
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int t = n % 2 * 8 + lane / 4, c = lane % 4 * 8;
            const uint4 v = *reinterpret_cast<const uint4*>(tile + (n / 2 * 16 + t) * LD + c);
            if (tb * 16 + t >= nt) continue;
            IO* o = static_cast<IO*>(n < 2 ? a.dr : a.dk) + rows + (tb * 16 + t) * vs + i0 + c;
            if (a.vec) {
                *reinterpret_cast<uint4*>(o) = v;
            } else {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    reinterpret_cast<unsigned short*>(o)[i] = static_cast<unsigned short>(w[i / 2] >> (16 * (i & 1)));
            }
        }
    }
}

// A segment token by token, in which something is not finite: its products by
// blocks met the zeros of tokens that it must not reach.  dr, dk and dw are written
// again; e, du (the walks') and dvv are right.  A thread holds a quarter of a key's
// row of the states.  smem: the segment's tiles, which are over.  False, and nothing
// is done, where the products are right: a state that enters as not finite leaves
// nothing finite, and a gradient of the last state that is not finite nothing of dk
// and dw (odd_dr: something in this thread's dr is not finite).
//   forward   S_t, dr_t = S_t dy_t, the part -a_t S_{t-1} dv_t of dk_t, and m, the
//             last token that leaves a finite state
//   backward  D_t, the part D_t u_t of dk_t, and <D, S> behind token m, where the
//             sums that dw takes may begin: of tokens behind m + 1 there is none
template <typename IO, int N>
__device__ __forceinline__ bool segment_tokens(const Args& a, const Segment& sg, char* smem, const float* s_seg, const float* d_seg,
                                               const float* dvv, bool odd_dr, int tid) {
    constexpr int J = N / 4, WARPS = 4 * N / 32;   // four threads a key
    float* dkp = reinterpret_cast<float*>(smem);      // (tokens, N)
    float* rdr = dkp + kSegment * N;                  // (tokens, warps)
    float* sum = rdr + kSegment * WARPS;              // (2, warps)
    int& bad = *reinterpret_cast<int*>(sum + 2 * WARPS);   // the first token whose state is not finite
    const int i = tid / 4, j = tid % 4 * J, lane = tid % 32, warp = tid / 32, nt = sg.nt;
    const bool whole = a.H == a.Hk;
    const auto entry = [&](const float* s, int q) { return s[kTcSegments<IO, N> ? i * N + j + q : (j + q) * N + i]; };
    const auto key = [&](const void* x, int t) { return to_f32(static_cast<const IO*>(x)[sg.keys + t * sg.ks + i]); };
    const auto fade = [&](int t) { return expf(-a.w[sg.scalar + t * a.H]); };
    const auto value = [&](const float* x, int t, int q) { return a.beta[sg.scalar + t * a.H] * x[sg.rows + t * sg.vs + j + q]; };
    const auto dy = [&](int t, int q) { return to_f32(static_cast<const IO*>(a.dy)[sg.rows + t * sg.vs + j + q]); };
    const auto out = [&](void* x, float* h, int t, float v) {
        const int64_t at = sg.rows + t * sg.vs + i;
        if (whole) put(static_cast<IO*>(x) + at, v);
        else h[at] = v;
    };
    float S[J], D[J], z[2] = {0.f, 0.f};   // z: NaN where S, D are not finite
#pragma unroll
    for (int q = 0; q < J; ++q) {
        S[q] = entry(s_seg, q);
        z[0] = fmaf(S[q], 0.f, z[0]);
        z[1] = fmaf(entry(d_seg, q), 0.f, z[1]);
    }
    const bool s_odd = __syncthreads_or(z[0] != 0.f), d_odd = __syncthreads_or(z[1] != 0.f);
    if (s_odd || (d_odd && !__syncthreads_or(odd_dr))) return false;
    if (tid == 0) bad = nt;
    __syncthreads();
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
        const float f = fade(t), k = key(a.k, t);
        float x = 0.f, z = 0.f, odd = 0.f;
#pragma unroll
        for (int q = 0; q < J; ++q) {
            S[q] *= f;
            x = fmaf(S[q], value(a.du, t, q), x);
            S[q] = fmaf(k, value(a.e, t, q), S[q]);
            z = fmaf(S[q], dy(t, q), z);
            odd = fmaf(S[q], 0.f, odd);
        }
        if (odd != 0.f) atomicMin(&bad, t);
        x = quad_sum(x), z = quad_sum(z);
        float p = lane % 4 == 0 ? key(a.r, t) * z : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o /= 2) p += __shfl_xor_sync(0xffffffffu, p, o);
        if (lane == 0) rdr[t * WARPS + warp] = p;
        if (lane % 4 == 0) {
            dkp[t * N + i] = -x;
            out(a.dr, a.drh, t, z);
        }
    }
    __syncthreads();
    const int m = bad - 1;
#pragma unroll
    for (int q = 0; q < J; ++q) S[q] = entry(s_seg, q), D[q] = entry(d_seg, q);
#pragma unroll 1
    for (int t = 0; t <= m; ++t) {
        const float f = fade(t), k = key(a.k, t);
#pragma unroll
        for (int q = 0; q < J; ++q) S[q] = fmaf(k, value(a.e, t, q), f * S[q]);
    }
    const auto inner = [&](int to) {   // of the state at hand and D
        float x = 0.f;
#pragma unroll
        for (int q = 0; q < J; ++q) x = fmaf(S[q], D[q], x);
#pragma unroll
        for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) sum[to * WARPS + warp] = x;
    };
#pragma unroll 1
    for (int t = nt - 1; t >= 0; --t) {
        if (t == m) inner(0);
        const float f = fade(t), k = key(a.k, t), r = key(a.r, t);
        float x = 0.f;
#pragma unroll
        for (int q = 0; q < J; ++q) {
            D[q] = fmaf(r, dy(t, q), D[q]);
            x = fmaf(D[q], value(a.e, t, q), x);
            D[q] = f * fmaf(k, -value(a.du, t, q), D[q]);
        }
        x = quad_sum(x);
        if (lane % 4 == 0) out(a.dk, a.dkh, t, x + dkp[t * N + i]);
    }
    if (m < 0) inner(0);
#pragma unroll
    for (int q = 0; q < J; ++q) S[q] = entry(s_seg, q);
    inner(1);
    __syncthreads();
    if (tid == 0) {
        float phi = 0.f, begin = 0.f;   // <D, S> behind token t, ahead of the first
        for (int w = 0; w < WARPS; ++w) phi += sum[w], begin += sum[WARPS + w];
#pragma unroll 1
        for (int t = nt - 1; t >= 0; --t) {
            const bool reset = fade(t) == 0.f;
            float g = t > m + 1 ? __int_as_float(0x7fffffff) : phi;
            if (t <= m) {
                float p = -dvv[t];
                for (int w = 0; w < WARPS; ++w) p += rdr[t * WARPS + w];
                g += p;
            }
            if (reset) g = 0.f;
            if (t <= m) phi = g;
            a.dw[sg.scalar + t * a.H] = -(t == 0 && !reset ? begin : g);
        }
    }
    return true;
}

// Is one of these not finite, or their sum?  (A sum of finite values that is not
// costs its segment time and nothing else.)
template <int NP>
__device__ __forceinline__ bool any_odd(const float (&x)[NP][2][4]) {
    F2 s = f2s(0.f);
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; i += 2) s = add2(s, f2(x[p][n][i], x[p][n][i + 1]));
    return !(fabsf(f2lo(s) + f2hi(s)) <= 3.4e38f);
}

// dw of a segment from r . dr by the warps' rows (own), dv . v and <D, S> at its
// end (border[1], a thread's share); rates: warp 0's, of two tokens a lane.  All
// threads of the CTA.  <D, S> at its begin follows from those, but in the first
// segment it is formed too: with an empty state it is zero, and not what rounding
// leaves of the terms.  At a token whose
// decay is 0 the sum is 0 and begins anew, so that what rounding leaves of the
// terms behind it does not reach the document ahead of it.
// odd_dr, odd_dk: something in this thread's is not finite; smem: the segment's tiles.
template <typename IO, int N, int PARTS>
__device__ __forceinline__ void segment_rates(const Args& a, const Segment& sg, float (&own)[2], float (&border)[2], float* rdr,
                                              const float* dvv, float* inner, const float* s_seg, const float* d_seg, int t_lo, float2 rates,
                                              bool odd_dr, bool odd_dk, char* smem, int tid) {
    constexpr int WARPS = 4 * PARTS, THREADS = 32 * WARPS;
    static_assert(THREADS == 4 * N, "segment_tokens' threads");
    const int lane = tid % 32, warp = tid / 32, nt = sg.nt;
    const int64_t scalar = sg.scalar, seg = sg.seg;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        own[q] += __shfl_xor_sync(0xffffffffu, own[q], 1);
        own[q] += __shfl_xor_sync(0xffffffffu, own[q], 2);
        if (lane % 4 == 0) rdr[(warp / 4) * kSegment + t_lo + 8 * q] = own[q];
    }
    if (seg == 0) {
        const float4* ps = reinterpret_cast<const float4*>(s_seg);
        const float4* pd = reinterpret_cast<const float4*>(d_seg - N * N);
#pragma unroll 4
        for (int i = tid; i < N * N / 4; i += THREADS) {
            const float4 u = __ldcg(ps + i), v = __ldcg(pd + i);
            border[0] = fmaf(u.x, v.x, fmaf(u.y, v.y, fmaf(u.z, v.z, fmaf(u.w, v.w, border[0]))));
        }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int o = 16; o > 0; o /= 2) border[q] += __shfl_xor_sync(0xffffffffu, border[q], o);
    if (lane == 0) inner[2 * warp] = border[0], inner[2 * warp + 1] = border[1];
    if (__syncthreads_or(odd_dr || odd_dk) && segment_tokens<IO, N>(a, sg, smem, s_seg, d_seg, dvv, odd_dr, tid)) return;
    // --- dw: the sum <Dn, S> from the segment's end backwards
    if (warp == 0) {
        float first = 0.f, end = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) first += inner[2 * i], end += inner[2 * i + 1];
        const int ta = 2 * lane;
        float term[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int t = ta + q;
            float x = rdr[t];
#pragma unroll
            for (int p = 1; p < PARTS; ++p) x += rdr[p * kSegment + t];
            term[q] = t < nt ? x - dvv[t] : 0.f;
        }
        // suffix sums over the lanes, each to the first reset
        const bool r0 = expf(-rates.x) == 0.f, r1 = expf(-rates.y) == 0.f;
        float x = r0 ? 0.f : r1 ? term[0] : term[0] + term[1];
        int cut = r0 || r1;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const float y = __shfl_down_sync(0xffffffffu, x, o);
            const int c = __shfl_down_sync(0xffffffffu, cut, o);
            if (lane + o < 32) {
                if (!cut) x += y;
                cut |= c;
            }
        }
        float after = __shfl_down_sync(0xffffffffu, x, 1);
        const int far = __shfl_down_sync(0xffffffffu, cut, 1);
        if (lane == 31) after = 0.f;
        else if (far) end = 0.f;
        const float s1 = r1 ? 0.f : end + (after + term[1]);
        const float s0 = r0 ? 0.f : r1 ? term[0] : end + (after + (term[1] + term[0]));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int t = ta + q;
            if (t >= nt) continue;
            const int64_t at = scalar + t * a.H;
            a.dw[at] = t == 0 && seg == 0 && !r0 ? -first : -(q ? s1 : s0);
        }
    }
}

template <typename IO, int N>
__global__ void __launch_bounds__(SegmentShape<IO, N>::THREADS, SegmentShape<IO, N>::CTAS) delta_segment_kernel(const Args a) {
    using G = SegmentShape<IO, N>;
    constexpr int KP = G::KP, NP = G::IC / 16;
    constexpr Swizzled<N> place{};
    extern __shared__ __align__(128) char swizzled_smem[];        // gram_at's exclusive or is of addresses
    char* const smem = swizzled_smem;
    __nv_bfloat16* ub = reinterpret_cast<__nv_bfloat16*>(smem);   // u = beta e
    __nv_bfloat16* db = ub + 3 * G::PIECE;                        // dv = beta du
    __nv_bfloat16* yb = db + 3 * G::PIECE;
    __nv_bfloat16* buf = reinterpret_cast<__nv_bfloat16*>(smem + G::S_ROWS);
    __nv_bfloat16* kb = KP == 1 ? reinterpret_cast<__nv_bfloat16*>(smem + G::S_ROWS + G::S_BUF) : ub;
    __nv_bfloat16* rb = kb + KP * G::PIECE;
    float2* sums = reinterpret_cast<float2*>(smem + G::S_ROWS + G::S_BUF + G::S_KEYS);
    float* dvv = reinterpret_cast<float*>(sums + kSegment);       // dv . v of a token
    float* rdr = dvv + kSegment;                                  // r . dr, by parts of the channels
    float* inner = rdr + kSegment * G::PARTS;                    // <D, S> at the borders, by warps
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int tb = warp % 4, i0 = warp / 4 * G::IC;

    const Segment sg(a, N, blockIdx.x);

    pdl_wait();

    // what is read later, on its way to L2 now
    const float* s_seg = a.s_seg + sg.state;
    const float* d_seg = a.d_seg + sg.state + N * N;
    const IO* kp = static_cast<const IO*>(a.k) + sg.keys;
    const IO* rp = static_cast<const IO*>(a.r) + sg.keys;
    for (int i = G::JB * N / 32 + tid; i < N * N / 32; i += G::THREADS) {
        prefetch_l2(s_seg + i * 32);
        prefetch_l2(s_seg + N * N + i * 32);
        prefetch_l2(d_seg + i * 32);
    }
    constexpr int LW = G::JB / G::WARPS, LU = LW * N / 128;   // lines of S and D of a warp, and its loads
    float4 ls[LU], ld[LU], le[LU];                            // S, D, S at the segment's end
    const auto load_lines_at = [&](int jb) {
#pragma unroll
        for (int u = 0; u < LU; ++u) {
            const int at = (jb + warp * LW) * N + (lane + u * 32) * 4;
            ls[u] = load4(s_seg + at, true);
            ld[u] = load4(d_seg + at, true);
            le[u] = load4(s_seg + N * N + at, true);
        }
    };
    load_lines_at(0);

    // --- the segment's rows: 16 / PARTS a warp
    constexpr int RW = 16 / G::PARTS;
    const int row = warp * RW, left = sg.nt - row;
    const int64_t rr = left > 0 ? row : 0;   // rows behind the last token: zeros, addressed at one that exists
    const auto rows_at = [&](int r, int c) { return place(row + r, c); };
    if constexpr (KP == 1) {
        copy_rows<IO, RW, N>(reinterpret_cast<IO*>(yb), rows_at, static_cast<const IO*>(a.dy) + sg.rows + rr * sg.vs, sg.vs, left, a.vec, lane);
        copy_rows<IO, RW, N>(reinterpret_cast<IO*>(kb), rows_at, kp + rr * sg.ks, sg.ks, left, a.vec, lane);
        copy_rows<IO, RW, N>(reinterpret_cast<IO*>(rb), rows_at, rp + rr * sg.ks, sg.ks, left, a.vec, lane);
        cp_async_commit();
    }
    stage_values<IO, N, RW>(a, sg, ub, db, G::PIECE, place, row, dvv, lane);
    if constexpr (KP == 3)
        split_rows<RW, N, 3>(yb, rows_at, G::PIECE, reinterpret_cast<const float*>(a.dy) + sg.rows + rr * sg.vs, sg.vs, left, a.vec, lane);
    const float2 rates = warp == 0 ? segment_sums(a, sg, sums, lane) : make_float2(0.f, 0.f);

    float border[2] = {0.f, 0.f};
    // --- the products with S and D: C[t][i], tiles of 16 channels
    float dr[NP][2][4], dk[NP][2][4];
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) dr[p][n][i] = dk[p][n][i] = 0.f;
    // this lane's places (bytes): as an A operand or a transposed B, and as a plain B; the columns' by exclusive or
    const uint32_t at_t = place((lane & 7) + ((lane >> 3) & 1) * 8, (lane >> 4) * 8) * 2;
    const uint32_t at_p = place((lane & 7) + (lane >> 4) * 8, ((lane >> 3) & 1) * 8) * 2;
    constexpr int PB = G::PIECE * 2, SB = G::SPIECE * 2, ROWS16 = 16 * N * 2;
    const uint32_t ub_a = smem_u32(ub), db_a = ub_a + 3 * PB, yb_a = db_a + 3 * PB, buf_a = ub_a + G::S_ROWS,
                   kb_a = KP == 1 ? buf_a + G::S_BUF : ub_a;
    const uint32_t own_a = ub_a + tb * ROWS16, at_i = at_t ^ (i0 * 2);   // the warp's tokens, its channels
    const int t_lo = tb * 16 + lane / 4;                  // this lane's rows: t_lo and t_lo + 8
    float2 gq[2];   // of the lane's two rows: g, q
#pragma unroll 1
    for (int jb = 0; jb < N; jb += G::JB) {
        if (jb > 0) __syncthreads();
#pragma unroll
        for (int u = 0; u < LU; ++u) {
            const int i = lane + u * 32, at = place(warp * LW + i / (N / 4), i % (N / 4) * 4);
            put4<3>(buf + at, G::SPIECE, ls[u]);
            put4<3>(buf + 3 * G::SPIECE + at, G::SPIECE, ld[u]);
            border[1] += fmaf(ld[u].x, le[u].x, ld[u].y * le[u].y) + fmaf(ld[u].z, le[u].z, ld[u].w * le[u].w);
        }
        if (KP == 1 && jb == 0) cp_async_wait();
        __syncthreads();
        if (jb + G::JB < N) load_lines_at(jb + G::JB);
        if (jb == 0) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                gq[q] = make_float2(decay_of(sums[t_lo + 8 * q], make_float2(0.f, 0.f)), decay_of(sums[kSegment - 1], sums[t_lo + 8 * q]));
        }
        const uint32_t col = at_t ^ (jb * 2);
        add_lines<N, KP, 3, 3>(dr, gq[0].x, gq[1].x, own_a + 6 * PB, PB, col, buf_a, SB, at_i);
        add_lines<N, 3, 3, 3>(dk, -gq[0].x, -gq[1].x, own_a + 3 * PB, PB, col, buf_a, SB, at_i);
        add_lines<N, 3, 3, 3>(dk, gq[0].y, gq[1].y, own_a, PB, col, buf_a + 3 * SB, SB, at_i);
    }

    // --- the blocks of token pairs s <= t, with the decays between the tokens: dy_t.u_s, and
    // -dv_t.u_s for s < t
    __syncthreads();
#pragma unroll 1
    for (int task = warp; task < 2 * G::BLOCKS; task += G::WARPS) {
        const int blk = task >> 1, bt = blk < 1 ? 0 : blk < 3 ? 1 : blk < 6 ? 2 : 3, bs = blk - bt * (bt + 1) / 2;
        const bool ofv = task & 1;
        __nv_bfloat16* m = buf + (blk * G::MATS + (ofv ? 3 : 0)) * kMat;
        const uint32_t xt = bt * ROWS16 + at_t, ys = ub_a + bs * ROWS16 + at_p;
        const int far = (bt > bs ? kChunk : 0) - ofv;   // s <= t + far
        float x[2][4];
        if (ofv) gram_at<N, 3, 3, 3, kChain<IO>, true>(x, db_a + xt, ys, PB);
        else gram_at<N, KP, 3, 3, kChain<IO>, true>(x, yb_a + xt, ys, PB);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int t = lane / 4 + 8 * q, c = 8 * n + 2 * (lane % 4);
                const float2 wt = sums[bt * 16 + t], w0 = sums[bs * 16 + c], w1 = sums[bs * 16 + c + 1];
                const float y0 = c <= t + far ? decay_of(wt, w0) * x[n][2 * q] : 0.f;
                const float y1 = c + 1 <= t + far ? decay_of(wt, w1) * x[n][2 * q + 1] : 0.f;
                put_pieces<3>(m, t, c, ofv ? -y0 : y0, ofv ? -y1 : y1);
            }
    }
    __syncthreads();
    if constexpr (KP == 3) {   // K and R over the rows
        split_rows<RW, N, 3>(kb, rows_at, G::PIECE, reinterpret_cast<const float*>(kp) + rr * sg.ks, sg.ks, left, a.vec, lane);
        split_rows<RW, N, 3>(rb, rows_at, G::PIECE, reinterpret_cast<const float*>(rp) + rr * sg.ks, sg.ks, left, a.vec, lane);
        __syncthreads();
    }
    // dr takes K by the rows of the blocks, dk K by rows and columns and R by columns
    const auto times_add = [&](float (&d)[2][4], const uint32_t (&a)[3][4], const uint32_t (&f)[KP][4]) {
        float x[2][4];
        times_sum<3, KP, 3>(x, true, a, f);
        Acc::add(d, x, false);
    };
#pragma unroll 1
    for (int sb = 0; sb < 4; ++sb) {
        const bool low = sb <= tb, up = sb >= tb;
        uint32_t dq[3][4], kq[3][4], rq[3][4], kt[3][4];
        if (low) {
            const uint32_t m = buf_a + ((tb * (tb + 1) / 2 + sb) * G::MATS * kMat + m_trans(lane)) * 2;
#pragma unroll
            for (int c = 0; c < 3; ++c) ldsm4(dq[c], m + c * kMat * 2);
#pragma unroll
            for (int c = 0; c < 3; ++c) ldsm4(kq[c], m + (3 + c) * kMat * 2);
        }
        if (up) {
            const uint32_t m = buf_a + ((sb * (sb + 1) / 2 + tb) * G::MATS * kMat + m_plain(lane)) * 2;
#pragma unroll
            for (int c = 0; c < 3; ++c) {
                ldsm4t(rq[c], m + c * kMat * 2);
                ldsm4t(kt[c], m + (3 + c) * kMat * 2);
            }
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const uint32_t so = kb_a + sb * ROWS16 + (at_t ^ ((i0 + p * 16) * 2));
            uint32_t fk[KP][4];
#pragma unroll
            for (int c = 0; c < KP; ++c) ldsm4t(fk[c], so + c * PB);
            if (low) {
                times_add(dr[p], dq, fk);
                times_add(dk[p], kq, fk);
            }
            if (up) {
                uint32_t fr[KP][4];
#pragma unroll
                for (int c = 0; c < KP; ++c) ldsm4t(fr[c], so + (KP + c) * PB);
                times_add(dk[p], kt, fk);
                times_add(dk[p], rq, fr);
            }
        }
    }
    float own[2];
    row_products<N, NP, KP>(own, rb, G::PIECE, dr, t_lo, i0, lane);
    store_rows<IO, N, NP>(a, sg, dr, dk, ub + warp * 2 * 16 * (G::IC + 8), tb, i0, lane);
    segment_rates<IO, N, G::PARTS>(a, sg, own, border, rdr, dvv, inner, s_seg, d_seg, t_lo, rates, any_odd(dr), any_odd(dk), smem, tid);
}

// dr and dk of a key head: the sums over the value heads that share it, in
// their order.  One thread per 4 channels.
template <typename IO, int N>
__global__ void __launch_bounds__(256) delta_share_kernel(const Args a) {
    const int64_t id = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    pdl_wait();
    if (id >= a.B * a.T * a.Hk * (N / 4)) return;
    const int64_t key = id / (N / 4);   // (sequence, token, key head)
    const int share = int(uint32_t(a.H) / uint32_t(a.Hk)), c = int(id % (N / 4)) * 4;
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

}  // namespace delta
}  // namespace wkv
