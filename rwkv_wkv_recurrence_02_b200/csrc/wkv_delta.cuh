// wkv_delta.cuh -- the gated delta rule: definitions and the kernels that work
// token by token.
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
// wkv_delta_mma.cuh has the forward walk, wkv_delta_mma_bwd.cuh the reverse
// mode; here is the single-token step.
#pragma once

#include "wkv_common.cuh"

namespace wkv {
namespace delta {

// tokens of a segment: the reverse mode keeps the states between segments
constexpr int kSegment = 64;
template <typename IO>
__device__ __forceinline__ float to_f32(IO x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// A workspace's first words; the error is where wkv_workspace_status() reads it,
// and these kernels write the last two only.
struct Control {
    uint32_t epoch, finished, error, err_unit;
};

// A wait ran out: in the call's workspace, and for the whole device (a call's
// workspace may be gone when somebody asks).
static __device__ uint32_t g_lost;
__device__ __forceinline__ void record_lost(Control* c, uint32_t unit) {
    c->error = 1u;
    c->err_unit = unit;
    g_lost = 1u;
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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
    // reverse mode's outputs
    void* dr;            // (B, T, Hk, N)
    void* dk;
    float* dw;           // (B, T, H)
    float* dbeta;
    // its workspace
    float* e;            // (B, T, H, N)
    float* du;
    float* s_seg;        // (B, H, n + 1, N, N), n = ceil(T / kSegment): the state entering each segment and the last (keep_state)
    float* d_seg;        // gradients of those, of what follows
    float* drh;          // (B, T, H, N): dr and dk of each value head, where heads share keys
    float* dkh;
    bool vec;            // 16-byte loads of every tensor in the I/O type
    // the error word, and the limit of waits
    Control* control;
    uint64_t wait_ns;
    // a walk in parts of part_len tokens, taken by tickets (parts > 1)
    int64_t parts, part_len;
    uint32_t* ticket;
    uint32_t* done;      // (walks): parts that are done
    float* hand;         // (B, H, N, N): the state between a walk's parts, as its warps hold it
};

// ---------------------------------------------------------------------------
// One token for L layers (B sequences, H heads each): the state is read once,
// held in registers and written once, which is what bounds it: 24 layers of 256
// sequences of 64 heads of 64 in 2244 us, 5.8 TB/s (90% of a copy's rate).  A warp
// takes CW value columns of a head; the sums over keys are shuffles.
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
    // 32-bit divisions: 2^32 heads' states would be 16 TB
    const uint32_t h32 = uint32_t(hh), H32 = uint32_t(H), row0 = h32 / H32;
    const int64_t hk = int64_t(row0) * Hk + (h32 - row0 * H32) / (H32 / uint32_t(Hk));
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
