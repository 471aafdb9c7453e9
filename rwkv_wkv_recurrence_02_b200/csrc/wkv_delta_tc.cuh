// wkv_delta_tc.cuh -- dr, dk, dbeta and dw of one segment of 64 tokens of the
// gated delta rule's reverse mode (wkv_delta_mma_bwd.cuh has the formulas), heads
// of 64 in bfloat16, with tcgen05.mma: every product is 64 x 64 x 64, one thread
// issues them, the accumulators are in tensor memory.
//
//   batch 1  Y S, V S, U D      rows of dy, dv, u with the states' keys
//            Y U^T              scores dy_t.u_s
//   batch 2  V U^T, U V^T       dv_t.u_s (s < t), u_t.dv_s (s > t)
//            U Y^T              u_t.dy_s
//   batch 3  A K (dr), B K + C R (dk): A, B, C the scores of tokens on their own
//            sides of the diagonal, with the decays between them
//
// Operands are bfloat16 pieces (dy, k and r exact, all others three), products of
// pieces smallest first into one accumulator, as many as the mma.sync form takes.
// K and R, whose tiles lie where D was, come in under batch 2.  All tiles are K-major without swizzle: 16-byte slots of 8 values,
// core matrices of 8 rows; a slot of padding behind each pair of core matrices and
// two behind each k step keep the stores of a warp in different banks.
//
// Measured for 8 x 2048 tokens of 32 heads (8192 segments), the whole call: 885 us, with the
// segments by mma.sync 929; on 8 x 4096 tokens 1735 us against 1837.  What bounds it is a
// CTA's chain at two CTAs an SM, about 27,700 cycles: loads and their conversion
// 6,700, the three batches 5,700, 5,500 and 2,600 (42 products; an M = 64 product of 16
// columns reads 4 KB of shared memory, and the CTA beside it wants the same unit, which
// is active in 48% of the cycles), scores 2,100 and 2,300, outputs 2,900; DRAM is at
// 24%, issue at 37%.  Steps, as the whole call's time when dk took 27 products: heads before segments in the grid's order (neighbours in
// memory at the same time) 1665 to 1637, descriptors by sums 1637 to 1617, dw's rates
// kept from the decays' sums 1617 to 1600, the next CTA's data prefetched while
// batch 1 runs 1600 to 1587 (with the CTA's own loads: no gain), 32-bit divisions
// for the CTA's place 1581 to 1542.  The scores' batch
// first, with S and D staged under it, was slower (413 against 408 us of this
// kernel), and so were more loads in flight (405 against 395).
#pragma once

#include "wkv_chunk.cuh"
#include "wkv_delta_mma_bwd.cuh"

namespace wkv {
namespace delta {

struct TcSegment {
    static constexpr int N = 64, THREADS = 256, PARTS = 2;
    static constexpr uint32_t LBO = 9, SBO = 17, KS = 138;      // slots: core matrices of a k step, row groups, k steps
    static constexpr uint32_t TILE = (3 * KS + 8 * SBO) * 16;   // bytes of 64 x 64 values
    // tiles: u (3), dv (3), dy; S (3), D (3).  Later C over u, B over dv, A over S;
    // over D first K, then R as they come (RAW), and K^T and R^T
    static constexpr int U = 0, V = 3, Y = 6, S = 7, D = 10, RAW = 12, TILES = 13;
    static constexpr int SUMS = TILES * TILE;
    static constexpr int SMEM = SUMS + 64 * (8 + 4);
    // in the end the outputs' rows over C, and the sums over channels behind them
    static constexpr int ROWS = 8 * 2 * 16 * 40;                // elements
    static_assert(ROWS * 2 + 64 * 8 + 64 <= 3 * int(TILE) && 64 * 64 * 2 <= int(TILE), "room in what is over");
    static constexpr uint32_t COLS = 256;                       // tensor memory: four accumulators
    // D fp32, A and B bfloat16, both K-major, N = 64, M = 64
    static constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((64u >> 3) << 17) | ((64u >> 4) << 24);
    static_assert(2 * (SMEM + 64 + 1024) <= 228 * 1024, "two CTAs an SM");
    // element offset of (row, k)
    __device__ __forceinline__ int operator()(int row, int k) const {
        return ((k >> 4) * KS + (row >> 3) * SBO + ((k >> 3) & 1) * LBO + (row & 7)) * 8 + (k & 7);
    }
};

__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
    return uint64_t((addr >> 4) & 0x3fffu) | uint64_t(TcSegment::LBO) << 16 | uint64_t(TcSegment::SBO) << 32 | uint64_t(1) << 46;
}
// d (+)= A B^T, a and b the tiles' descriptors (one thread).  A descriptor's
// address is its low field, in slots: those of other tiles and k steps are sums.
__device__ __forceinline__ void tile_product(uint32_t d, uint64_t a, uint64_t b, bool first) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a + TcSegment::KS * s), "l"(b + TcSegment::KS * s), "r"(TcSegment::IDESC), "r"(first && s == 0 ? 0u : 1u)
            : "memory");
}
__device__ __forceinline__ void tile_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// d = the products of two operands' three pieces, the first ones' descriptors
// given, smallest orders first
__device__ __forceinline__ void piece_products(uint32_t d, uint64_t a, uint64_t b) {
    constexpr int TILE = TcSegment::TILE / 16;
#pragma unroll
    for (int o = 2; o >= 0; --o)
#pragma unroll
        for (int p = o; p >= 0; --p) tile_product(d, a + p * TILE, b + (o - p) * TILE, o == 2 && p == 2);
}
// what every thread wrote to shared memory or read of tensor memory, before the next batch
__device__ __forceinline__ void before_batch() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Did a batch come in time?  Every thread of the CTA; its accumulators may be read
// then.  If not, the batch is waited for once more (it reads the tiles and writes
// tensor memory), the error word is set, and the CTA ends.  A limit of 0 asks once.
__device__ __forceinline__ bool batch_done(const Args& a, uint64_t* bar) {
    const bool mine = a.wait_ns > 0 ? mbar_wait(bar, 0, a.wait_ns) : mbar_test(bar, 0);
    const bool all = __syncthreads_and(mine);
    if (!all) {
        mbar_wait(bar, 0, kCopyWaitNs);
        if (threadIdx.x == 0) record_lost(a.control, blockIdx.x);
        __syncthreads();
    }
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    return all;
}
__device__ __forceinline__ void free_columns(uint32_t acc, int warp) {   // after a barrier behind every warp's loads
    if (warp == 0) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(acc), "r"(TcSegment::COLS) : "memory");
    }
}
// NaN for dr, dk and dw of a segment whose products did not come
__device__ __forceinline__ void lose_segment(const Args& a, const Segment& sg, uint32_t acc, int tid) {
    const float bad = __int_as_float(0x7fffffff);
    for (int i = tid; i < sg.nt * TcSegment::N; i += TcSegment::THREADS) {
        const int64_t at = sg.rows + i / TcSegment::N * sg.vs + i % TcSegment::N;
        if (a.H == a.Hk) put(static_cast<__nv_bfloat16*>(a.dr) + at, bad), put(static_cast<__nv_bfloat16*>(a.dk) + at, bad);
        else a.drh[at] = a.dkh[at] = bad;
        if (i < sg.nt) a.dw[sg.scalar + i * a.H] = bad;
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    free_columns(acc, tid / 32);
}
// 16 rows x 32 columns of an accumulator: x[p][n][i] is row lane / 4 + 8 (i / 2),
// column 16 p + 8 n + 2 (lane % 4) + i % 2
__device__ __forceinline__ void load_tile(uint32_t addr, float (&x)[2][2][4]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[g / 2][g % 2][i] = __uint_as_float(r[4 * g + i]);
}

// the CTA that follows this one on its SM, about: two CTAs on each of 148 SMs
constexpr int kAhead = 296;

__global__ void __launch_bounds__(TcSegment::THREADS, 2) delta_segment_tc_kernel(const Args a) {
    using G = TcSegment;
    using IO = __nv_bfloat16;
    constexpr int N = G::N, PC = G::TILE / 2;   // elements of a tile
    constexpr G at{};
    constexpr Swizzled<N> place{};
    extern __shared__ __align__(16) char smem[];
    __shared__ __align__(8) uint64_t bar[3];
    __shared__ uint32_t slot;
    __nv_bfloat16* tiles = reinterpret_cast<__nv_bfloat16*>(smem);
    __nv_bfloat16* raw = tiles + G::RAW * PC;
    float2* sums = reinterpret_cast<float2*>(smem + G::SUMS);
    float* dvv = reinterpret_cast<float*>(sums + kSegment);
    float* rdr = reinterpret_cast<float*>(tiles + G::U * PC + G::ROWS);
    float* inner = rdr + kSegment * G::PARTS;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    // the warp's tokens and channels (and, of scores, columns)
    const int tb = warp % 4, i0 = warp / 4 * 32, t_lo = tb * 16 + lane / 4;
    const Segment sg(a, N, blockIdx.x);

    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < 3; ++i) mbar_init(&bar[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&slot)), "r"(G::COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }

    pdl_wait();

    // --- all that comes from memory: a warp's 8 keys of S and D, its 8 tokens' rows
    const float* s_seg = a.s_seg + sg.state;
    const float* d_seg = a.d_seg + sg.state + N * N;
    float4 ls[2], ld[2], le[2];
    const auto load_lines_at = [&](int half) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int o = (warp * 8 + half * 4) * N + (lane + u * 32) * 4;
            ls[u] = load4(s_seg + o, true);
            ld[u] = load4(d_seg + o, true);
            le[u] = load4(s_seg + N * N + o, true);
        }
    };
    load_lines_at(0);
    const int row = warp * 8, left = sg.nt - row;
    const int64_t first = left > 0 ? row : 0;   // rows behind the last token: zeros, addressed at one that exists
    copy_rows<IO, 8, N>(tiles + G::Y * PC, [&](int r, int c) { return at(row + r, c); },
                        static_cast<const IO*>(a.dy) + sg.rows + first * sg.vs, sg.vs, left, a.vec, lane);
    cp_async_commit();
    stage_values<IO, N, 8>(a, sg, tiles + G::U * PC, tiles + G::V * PC, PC, at, row, dvv, lane);
    const float2 rates = warp == 0 ? segment_sums(a, sg, sums, lane) : make_float2(0.f, 0.f);
    float border[2] = {0.f, 0.f};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = lane + u * 32, o = at(warp * 8 + half * 4 + i / 16, i % 16 * 4);
            put4<3>(tiles + G::S * PC + o, PC, ls[u]);
            put4<3>(tiles + G::D * PC + o, PC, ld[u]);
            border[1] += fmaf(ld[u].x, le[u].x, ld[u].y * le[u].y) + fmaf(ld[u].z, le[u].z, ld[u].w * le[u].w);
        }
        if (half == 0) load_lines_at(1);
    }
    cp_async_wait();
    before_batch();

    const uint32_t acc = slot, mine = acc + (uint32_t(32 * tb) << 16) + i0;   // this warp's rows and columns
    const uint64_t t0 = tile_desc(smem_u32(tiles));
    const auto tile = [&](int i) { return t0 + i * (G::TILE / 16); };
    if (tid == 0) {
#pragma unroll
        for (int p = 2; p >= 0; --p) tile_product(acc, tile(G::Y), tile(G::S + p), p == 2);
        piece_products(acc + 64, tile(G::V), tile(G::S));
        piece_products(acc + 128, tile(G::U), tile(G::D));
#pragma unroll
        for (int p = 2; p >= 0; --p) tile_product(acc + 192, tile(G::Y), tile(G::U + p), p == 2);
        tile_commit(&bar[0]);
    }
    // what that CTA will read, on its way to L2
    {
        const Segment nx(a, N, int64_t(blockIdx.x) + kAhead);
        if (nx.head < a.B * a.H) {
            const float* lines[2] = {a.s_seg + nx.state, a.d_seg + nx.state + N * N};
            prefetch_l2(lines[tid / 128] + tid % 128 * 32);
            const int t = tid / 4;
            if (t < nx.nt) {
                prefetch_l2((tid & 2 ? a.du : a.e) + nx.rows + t * nx.vs + (tid & 1) * 32);
                prefetch_l2(static_cast<const IO*>(tid & 2 ? (tid & 1 ? a.k : a.r) : (tid & 1 ? a.v : a.dy)) +
                            (tid & 2 ? nx.keys + t * nx.ks : nx.rows + t * nx.vs));
            }
        }
    }
    float g[2], q[2];   // decays of the lane's two rows, up to them and after
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        g[h] = decay_of(sums[t_lo + 8 * h], make_float2(0.f, 0.f));
        q[h] = decay_of(sums[kSegment - 1], sums[t_lo + 8 * h]);
    }
    if (!batch_done(a, &bar[0])) return lose_segment(a, sg, acc, tid);
    // K, then R: a warp's 8 tokens as they come, later its 8 channels turned
    const auto fetch_raw = [&](const void* from) {
        copy_rows<IO, 8, N>(raw, [&](int r, int c) { return place(row + r, c); }, static_cast<const IO*>(from) + sg.keys + first * sg.ks,
                            sg.ks, left, a.vec, lane);
        cp_async_commit();
    };
    const auto turn_raw = [&](__nv_bfloat16* to) {   // 8 x 8 blocks turned on their way through registers
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t f[4];   // tokens 32 b .. 32 b + 31
            ldsm4t(f, smem_u32(raw + place(32 * b + lane, warp * 8)));
#pragma unroll
            for (int z = 0; z < 4; ++z)
                *reinterpret_cast<uint32_t*>(to + at(warp * 8 + lane / 4, 32 * b + 8 * z + 2 * (lane % 4))) = f[z];
        }
    };
    fetch_raw(a.k);
    float dr[2][2][4], dk[2][2][4], x[2][2][4];
    load_tile(mine, dr);
    load_tile(mine + 64, dk);
    load_tile(mine + 128, x);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dr[p][n][i] *= g[i >> 1];
                dk[p][n][i] = fmaf(q[i >> 1], x[p][n][i], -g[i >> 1] * dk[p][n][i]);
            }
    // A: dy_t.u_s, s <= t
    load_tile(mine + 192, x);
    const auto put_scores = [&](int t, int c, float y0, float y1, __nv_bfloat16* to) {
        uint32_t w[3];
        split2<3>(y0, y1, w);
#pragma unroll
        for (int z = 0; z < 3; ++z) *reinterpret_cast<uint32_t*>(to + z * PC + at(t, c)) = w[z];
    };
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = t_lo + 8 * h, c = i0 + 16 * p + 8 * n + 2 * (lane % 4);
                const float y0 = c <= t ? decay_of(sums[t], sums[c]) * x[p][n][2 * h] : 0.f;
                const float y1 = c + 1 <= t ? decay_of(sums[t], sums[c + 1]) * x[p][n][2 * h + 1] : 0.f;
                put_scores(t, c, y0, y1, tiles + G::S * PC);
            }
    cp_async_wait();
    before_batch();
    if (tid == 0) {
        piece_products(acc, tile(G::V), tile(G::U));
        piece_products(acc + 64, tile(G::U), tile(G::V));
#pragma unroll
        for (int p = 2; p >= 0; --p) tile_product(acc + 128, tile(G::U + p), tile(G::Y), p == 2);
        tile_commit(&bar[1]);
    }
    turn_raw(tiles + G::D * PC);
    __syncthreads();
    fetch_raw(a.r);
    cp_async_wait();
    __syncthreads();
    turn_raw(tiles + (G::D + 1) * PC);
    if (!batch_done(a, &bar[1])) return lose_segment(a, sg, acc, tid);
    // B: -dv_t.u_s, s < t, and -u_t.dv_s, s > t; C: u_t.dy_s, s >= t
    {
        float y[2][2][4], z[2][2][4];
        load_tile(mine, x);
        load_tile(mine + 64, y);
        load_tile(mine + 128, z);
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = t_lo + 8 * h, c = i0 + 16 * p + 8 * n + 2 * (lane % 4);
                    const float2 wt = sums[t];
                    float b[2], cc[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 ws = sums[c + e];
                        const bool below = c + e < t;
                        const float d = below ? decay_of(wt, ws) : decay_of(ws, wt);
                        b[e] = c + e == t ? 0.f : -d * (below ? x[p][n][2 * h + e] : y[p][n][2 * h + e]);
                        cc[e] = below ? 0.f : d * z[p][n][2 * h + e];
                    }
                    put_scores(t, c, b[0], b[1], tiles + G::V * PC);
                    put_scores(t, c, cc[0], cc[1], tiles + G::U * PC);
                }
    }
    before_batch();
    if (tid == 0) {
#pragma unroll
        for (int p = 2; p >= 0; --p) tile_product(acc, tile(G::S + p), tile(G::D), p == 2);
#pragma unroll
        for (int p = 2; p >= 0; --p) {
            tile_product(acc + 64, tile(G::V + p), tile(G::D), p == 2);
            tile_product(acc + 64, tile(G::U + p), tile(G::D + 1), false);
        }
        tile_commit(&bar[2]);
    }
    if (!batch_done(a, &bar[2])) return lose_segment(a, sg, acc, tid);
    load_tile(mine, x);
#pragma unroll
    for (int p = 0; p < 2; ++p) Acc::add(dr[p], x[p], false);
    load_tile(mine + 64, x);
#pragma unroll
    for (int p = 0; p < 2; ++p) Acc::add(dk[p], x[p], false);
    float own[2];
    row_products<N, 2, 1>(own, raw, 0, dr, t_lo, i0, lane);
    store_rows<IO, N, 2>(a, sg, dr, dk, tiles + G::U * PC + warp * (G::ROWS / 8), tb, i0, lane);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    segment_rates<IO, N, G::PARTS>(a, sg, own, border, rdr, dvv, inner, s_seg, d_seg, t_lo, rates, any_odd(dr), any_odd(dk), smem, tid);
    free_columns(acc, warp);   // every warp's loads are done: the barrier in segment_rates
}

}  // namespace delta
}  // namespace wkv
