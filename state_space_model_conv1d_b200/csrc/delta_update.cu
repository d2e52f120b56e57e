// delta_update.cu -- one token of the gated delta rule per batch row, in
// place on slot-indexed fp32 states.
//
//     w = a h,  u = beta (v - w . k),  h = w + u k,
//     y = scale (h . q) = scale (w . q + u (k . q))
//
// y in its second form needs no pass over the updated row, so both dot
// products are taken from one read and the row is written once: HBM-bound
// (8 bytes per state element).  8 lanes hold a state row (4 consecutive
// states of every 32: a row's 16-byte loads cover whole 128-byte lines), a
// warp four rows.  256 rows of 64 heads, P 64, N 128, bf16: 162 us for 1.08 GB,
// 6.7 TB/s.
#include "common.cuh"
#include "delta.h"

namespace ssm {
namespace {

constexpr int kThreads = 128;
constexpr int kStep = kThreads / 8;    // rows a CTA has in flight

// VEC: dstate % 4 == 0 (16-byte state accesses).  NV: 32-state runs per row.
template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(kThreads) delta_update_kernel(const ssm_delta_update_args a, int rows_per_cta) {
    const int64_t H = a.nheads, P = a.headdim, N = a.dstate;
    const int64_t b = blockIdx.y;
    const int h = blockIdx.x % (int)H;
    const int64_t p0 = (int64_t)(blockIdx.x / (int)H) * rows_per_cta, p1 = min(P, p0 + rows_per_cta);
    const int64_t slot = a.state_batch_indices ? a.state_batch_indices[b] : b;
    T *y = (T *)a.y + b * a.y_batch_stride + h * P;
    if (slot < 0 || slot >= a.nslots) {
        for (int64_t p = p0 + threadIdx.x; p < p1; p += kThreads) Elem<T>::st(y + p, 0.f);
        return;
    }
    const int lane8 = threadIdx.x & 7;
    const int64_t grp = h / (H / a.ngroups);
    const T *qp = (const T *)a.q + b * a.q_batch_stride + grp * N, *kp = (const T *)a.k + b * a.k_batch_stride + grp * N;
    const T *v = (const T *)a.v + b * a.v_batch_stride + h * P;
    float k[NV][4], q[NV][4], kq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = i * 32 + lane8 * 4 + e;
            k[i][e] = n < N ? Elem<T>::ld(kp + n) : 0.f;
            q[i][e] = n < N ? Elem<T>::ld(qp + n) : 0.f;
            kq = fmaf(k[i][e], q[i][e], kq);
        }
    kq += __shfl_xor_sync(~0u, kq, 1);
    kq += __shfl_xor_sync(~0u, kq, 2);
    kq += __shfl_xor_sync(~0u, kq, 4);
    const float al = decay_of(a.g[b * a.g_batch_stride + h]);
    const float be = a.beta[b * a.beta_batch_stride + h];
    float *st = a.state + ((slot * H + h) * P) * N;
    if (!SSM_BOUNDS((slot * H + h) * P + p1 - 1, a.nslots * H * P, BS_DELTA_STATE)) return;
    // every lane takes every turn, so that the shuffles see whole warps
    for (int64_t pb = p0; pb < p1; pb += kStep) {
        const int64_t p = pb + (threadIdx.x >> 3);
        const bool live = p < p1;
        float w[NV][4];
        float *row = st + p * N;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int n = i * 32 + lane8 * 4;
            if constexpr (VEC) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (live && n < N) x = __ldcs(reinterpret_cast<const float4 *>(row + n));
                w[i][0] = x.x; w[i][1] = x.y; w[i][2] = x.z; w[i][3] = x.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[i][e] = live && n + e < N ? row[n + e] : 0.f;
            }
        }
        const float vv = live ? Elem<T>::ld(v + p) : 0.f;
        float sk = 0.f, sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[i][e] *= al;
                sk = fmaf(w[i][e], k[i][e], sk);
                sq = fmaf(w[i][e], q[i][e], sq);
            }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            sk += __shfl_xor_sync(~0u, sk, o);
            sq += __shfl_xor_sync(~0u, sq, o);
        }
        const float u = be * (vv - sk);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int n = i * 32 + lane8 * 4;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[i][e] = fmaf(u, k[i][e], w[i][e]);
            if constexpr (VEC) {
                if (n < N) __stcs(reinterpret_cast<float4 *>(row + n), make_float4(w[i][0], w[i][1], w[i][2], w[i][3]));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < N) row[n + e] = w[i][e];
            }
        }
        if (lane8 == 0) Elem<T>::st(y + p, a.scale * fmaf(u, kq, sq));
    }
}

template <typename T, int NV>
void run(const ssm_delta_update_args &a, dim3 grid, int rows, cudaStream_t st) {
    if (a.dstate % 4 == 0) delta_update_kernel<T, NV, true><<<grid, kThreads, 0, st>>>(a, rows);
    else delta_update_kernel<T, NV, false><<<grid, kThreads, 0, st>>>(a, rows);
}
template <typename T>
void pick(const ssm_delta_update_args &a, dim3 grid, int rows, cudaStream_t st) {
    if (a.dstate <= 32) run<T, 1>(a, grid, rows, st);
    else if (a.dstate <= 64) run<T, 2>(a, grid, rows, st);
    else if (a.dstate <= 128) run<T, 4>(a, grid, rows, st);
    else run<T, 8>(a, grid, rows, st);
}

}  // namespace

cudaError_t launch_delta_update(const ssm_delta_update_args &a, cudaStream_t st) {
    if (a.batch == 0) return cudaSuccess;
    // 64 rows per CTA amortise the loads of k, q and the gates; with too few
    // (row, head) pairs to fill the GPU the rows are spread over more CTAs.  In us
    // with 64 / 16 rows: 256 x 64 heads of P 64 162 / 187, 16 x 32 of 64 7.2 / 8.5,
    // 3 x 32 of 128 5.6 / 4.7, 1 x 16 of 64 4.9 / 3.6 (N 128, bf16)
    int rows = 64;
    while (rows > kStep && a.batch * a.nheads * ((a.headdim + rows - 1) / rows) < 3LL * sm_count()) rows /= 2;
    const dim3 grid((unsigned)(a.nheads * ((a.headdim + rows - 1) / rows)), (unsigned)a.batch);
    timing_begin(st);
    if (a.dtype == SSM_BF16) pick<__nv_bfloat16>(a, grid, rows, st);
    else pick<float>(a, grid, rows, st);
    timing_end(st);
    return cudaGetLastError();
}

}  // namespace ssm
