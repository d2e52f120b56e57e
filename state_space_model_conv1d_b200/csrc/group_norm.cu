// group_norm.cu -- group norm of channels-last rows with an activation or a
// SiLU gate, forward and backward (formulas in ssm.h).
//
// A unit of TPU threads owns one group of every `stride`-th token and keeps
// the group in registers between the statistics and the output, so x (and z)
// are read once and y is written once: HBM-bound.  Units next to each other in
// a CTA own the groups next to each other of one token, so a CTA reads a
// contiguous stretch.  A unit stays with its group, which keeps the weights
// (forward) and their gradients' sums (backward) in registers over its tokens.
// Mean and M2 = sum (x - mean)^2 are merged pairwise (Chan's update) in one
// reduction: no cancellation however far the mean is from zero.
//
// Backward, with n the normalised values, t = n w + bias, dt = dL/dt, dn = dt w:
//     ds = r (dn - n mean(dn n) - [subtract_mean] mean(dn)),  r = 1/sqrt(var + eps)
//     dweight = sum_tokens dt n,  dbias = sum_tokens dt
// Each unit writes its sums over its tokens; a second kernel adds the units'
// shares in order.
#include "common.cuh"
#include "norm.h"

namespace ssm {
namespace {

struct Args {
    ssm_norm_args a;
    const void *dy;
    int64_t dy_bs, dy_ts;
    void *dx, *dz;
    float *pw, *pb;          // [splits][channels] shares of dweight, dbias
    int64_t rows;            // batch * seqlen
    int splits;              // units per group
};

// Sum of (n, mean, M2) triples over the unit's TPU threads; every thread gets
// the result.  `red` holds 3 floats per warp of the CTA.
SSM_DEVINL void merge(float &n, float &mean, float &m2, float nb, float mb, float m2b) {
    const float nn = n + nb;
    if (nn > 0.f) {
        const float d = mb - mean, f = nb / nn;
        m2 = m2 + m2b + d * d * n * f;
        mean = fmaf(d, f, mean);
    }
    n = nn;
}
template <int TPU>
SSM_DEVINL void unit_stats(float &n, float &mean, float &m2, float *red) {
#pragma unroll
    for (int o = 1; o < (TPU < 32 ? TPU : 32); o <<= 1) {
        const float nb = __shfl_xor_sync(~0u, n, o), mb = __shfl_xor_sync(~0u, mean, o),
                    m2b = __shfl_xor_sync(~0u, m2, o);
        merge(n, mean, m2, nb, mb, m2b);
    }
    if constexpr (TPU > 32) {
        const int warp = threadIdx.x >> 5, first = warp / (TPU / 32) * (TPU / 32);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
            red[3 * warp] = n;
            red[3 * warp + 1] = mean;
            red[3 * warp + 2] = m2;
        }
        __syncthreads();
        n = red[3 * first];
        mean = red[3 * first + 1];
        m2 = red[3 * first + 2];
#pragma unroll
        for (int i = 1; i < TPU / 32; ++i)
            merge(n, mean, m2, red[3 * (first + i)], red[3 * (first + i) + 1], red[3 * (first + i) + 2]);
    }
}
template <int TPU>
SSM_DEVINL void unit_sum2(float &u, float &v, float *red) {
#pragma unroll
    for (int o = 1; o < (TPU < 32 ? TPU : 32); o <<= 1) {
        u += __shfl_xor_sync(~0u, u, o);
        v += __shfl_xor_sync(~0u, v, o);
    }
    if constexpr (TPU > 32) {
        const int warp = threadIdx.x >> 5, first = warp / (TPU / 32) * (TPU / 32);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
            red[2 * warp] = u;
            red[2 * warp + 1] = v;
        }
        __syncthreads();
        u = v = 0.f;
#pragma unroll
        for (int i = 0; i < TPU / 32; ++i) {
            u += red[2 * (first + i)];
            v += red[2 * (first + i) + 1];
        }
    }
}

// Channel (within the group) of value e of vector i of this thread: runs of 8
// (16-byte accesses), or one channel per thread and step.
template <int TPU, bool VEC>
SSM_DEVINL int chan(int th, int i, int e) {
    return VEC ? (i * TPU + th) * 8 + e : (i * 8 + e) * TPU + th;
}
template <typename T, int TPU, int VPT, bool VEC>
SSM_DEVINL void load(float (&v)[VPT][8], const T *p, int th, int D) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (VEC) {
            if (chan<TPU, VEC>(th, i, 0) < D) Vec8<T>::ld(p + chan<TPU, VEC>(th, i, 0), v[i]);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = chan<TPU, VEC>(th, i, e);
                v[i][e] = c < D ? Elem<T>::ld(p + c) : 0.f;
            }
        }
    }
}
template <typename T, int TPU, int VPT, bool VEC>
SSM_DEVINL void store(T *p, const float (&v)[VPT][8], int th, int D) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (VEC) {
            if (chan<TPU, VEC>(th, i, 0) < D) Vec8<T>::st(p + chan<TPU, VEC>(th, i, 0), v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = chan<TPU, VEC>(th, i, e);
                if (c < D) Elem<T>::st(p + c, v[i][e]);
            }
        }
    }
}

SSM_DEVINL float sigmoid(float v) { return 1.f / (1.f + __expf(-v)); }

template <int TPU> constexpr int threads_of() { return TPU > 256 ? TPU : 256; }

// mean and 1 / sqrt(var + eps) of the group this unit holds in v
template <int TPU, int VPT, bool VEC>
SSM_DEVINL void stats(const float (&v)[VPT][8], int th, int D, bool centre, float eps, float *red, float &mean, float &r) {
    float n = 0.f, m2 = 0.f;
    mean = 0.f;
    if (centre) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (chan<TPU, VEC>(th, i, e) < D) {
                    s += v[i][e];
                    n += 1.f;
                }
        mean = n > 0.f ? s / n : 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (chan<TPU, VEC>(th, i, e) < D) m2 = fmaf(v[i][e] - mean, v[i][e] - mean, m2);
        unit_stats<TPU>(n, mean, m2, red);
    } else {
        float none = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) m2 = fmaf(v[i][e], v[i][e], m2);      // zeros past D
        unit_sum2<TPU>(m2, none, red);
    }
    r = 1.f / sqrtf(m2 / (float)D + eps);
}

template <typename T, int TPU, int VPT, bool VEC>
__global__ void __launch_bounds__(threads_of<TPU>()) group_norm_kernel(const Args p) {
    __shared__ float red[threads_of<TPU>() / 32 * 3];
    const ssm_norm_args &a = p.a;
    constexpr int UPB = threads_of<TPU>() / TPU;
    const int th = threadIdx.x % TPU, D = (int)(a.channels / a.groups);
    const int64_t unit = (int64_t)blockIdx.x * UPB + threadIdx.x / TPU;
    const int64_t grp = unit % a.groups, first = unit / a.groups;
    const int64_t c0 = grp * D;
    const bool gated = a.mode == SSM_NORM_GATE, pre = a.mode == SSM_NORM_GATE_FIRST, act = a.mode == SSM_NORM_SILU;
    float w[VPT][8], b[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = chan<TPU, VEC>(th, i, e);
            w[i][e] = a.weight && c < D ? a.weight[c0 + c] : 1.f;
            b[i][e] = a.bias && c < D ? a.bias[c0 + c] : 0.f;
        }
    // the same number of turns for every unit of a CTA: the sums of wide groups synchronise
    const int64_t turns = (p.rows + p.splits - 1) / p.splits;
    for (int64_t it = 0; it < turns; ++it) {
        const int64_t row = first + it * p.splits;
        const bool live = first < p.splits && row < p.rows;
        if (TPU <= 32 && __all_sync(~0u, !live)) break;
        const int64_t bi = live ? row / a.seqlen : 0, t = live ? row % a.seqlen : 0;
        float x[VPT][8], z[VPT][8];
        const int dl = live ? D : 0;
        load<T, TPU, VPT, VEC>(x, (const T *)a.x + bi * a.x_batch_stride + t * a.x_token_stride + c0, th, dl);
        if (gated || pre) load<T, TPU, VPT, VEC>(z, (const T *)a.z + bi * a.z_batch_stride + t * a.z_token_stride + c0, th, dl);
        if (pre)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] *= z[i][e] * sigmoid(z[i][e]);
        float mean, r;
        stats<TPU, VPT, VEC>(x, th, D, a.subtract_mean != 0, a.eps, red, mean, r);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = fmaf((x[i][e] - mean) * r, w[i][e], b[i][e]);
                if (gated) v *= z[i][e] * sigmoid(z[i][e]);
                if (act) v *= sigmoid(v);
                x[i][e] = v;
            }
        store<T, TPU, VPT, VEC>((T *)a.y + bi * a.y_batch_stride + t * a.y_token_stride + c0, x, th, D);
    }
}

template <typename T, int TPU, int VPT, bool VEC>
__global__ void __launch_bounds__(threads_of<TPU>()) group_norm_bwd_kernel(const Args p) {
    __shared__ float red[threads_of<TPU>() / 32 * 3];
    const ssm_norm_args &a = p.a;
    constexpr int UPB = threads_of<TPU>() / TPU;
    const int th = threadIdx.x % TPU, D = (int)(a.channels / a.groups);
    const int64_t unit = (int64_t)blockIdx.x * UPB + threadIdx.x / TPU;
    const int64_t grp = unit % a.groups, first = unit / a.groups;
    const int64_t c0 = grp * D;
    const bool gated = a.mode == SSM_NORM_GATE, pre = a.mode == SSM_NORM_GATE_FIRST, act = a.mode == SSM_NORM_SILU;
    const float inv = 1.f / (float)D;
    float w[VPT][8], b[VPT][8], dw[VPT][8], db[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = chan<TPU, VEC>(th, i, e);
            w[i][e] = a.weight && c < D ? a.weight[c0 + c] : 1.f;
            b[i][e] = a.bias && c < D ? a.bias[c0 + c] : 0.f;
            dw[i][e] = db[i][e] = 0.f;
        }
    const int64_t turns = (p.rows + p.splits - 1) / p.splits;
    for (int64_t it = 0; it < turns; ++it) {
        const int64_t row = first + it * p.splits;
        const bool live = first < p.splits && row < p.rows;
        if (TPU <= 32 && __all_sync(~0u, !live)) break;
        const int64_t bi = live ? row / a.seqlen : 0, t = live ? row % a.seqlen : 0;
        const int dl = live ? D : 0;
        float x[VPT][8], z[VPT][8], g[VPT][8], s[VPT][8];
        load<T, TPU, VPT, VEC>(x, (const T *)a.x + bi * a.x_batch_stride + t * a.x_token_stride + c0, th, dl);
        load<T, TPU, VPT, VEC>(g, (const T *)p.dy + bi * p.dy_bs + t * p.dy_ts + c0, th, dl);
        if (gated || pre) load<T, TPU, VPT, VEC>(z, (const T *)a.z + bi * a.z_batch_stride + t * a.z_token_stride + c0, th, dl);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[i][e] = pre ? x[i][e] * z[i][e] * sigmoid(z[i][e]) : x[i][e];
        float mean, r;
        stats<TPU, VPT, VEC>(s, th, D, a.subtract_mean != 0, a.eps, red, mean, r);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = chan<TPU, VEC>(th, i, e) < dl;
                const float n = in ? (s[i][e] - mean) * r : 0.f;
                float dt = g[i][e];
                if (gated || act) {
                    const float tt = fmaf(n, w[i][e], b[i][e]);
                    if (gated) {
                        const float sg = sigmoid(z[i][e]);
                        const float gate = z[i][e] * sg;
                        z[i][e] = dt * tt * fmaf(gate, 1.f - sg, sg);          // dz
                        dt *= gate;
                    } else {
                        const float sg = sigmoid(tt);
                        dt *= fmaf(tt * sg, 1.f - sg, sg);
                    }
                }
                s[i][e] = n;
                dw[i][e] = fmaf(dt, n, dw[i][e]);
                db[i][e] += dt;
                g[i][e] = dt * w[i][e];                                         // dn
                s1 += g[i][e];
                s2 = fmaf(g[i][e], n, s2);
            }
        unit_sum2<TPU>(s1, s2, red);
        if (!live) continue;
        s1 = a.subtract_mean ? s1 * inv : 0.f;
        s2 *= inv;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = r * (g[i][e] - s1 - s[i][e] * s2);
                if (pre) {
                    const float sg = sigmoid(z[i][e]);
                    const float gate = z[i][e] * sg;
                    z[i][e] = d * x[i][e] * fmaf(gate, 1.f - sg, sg);          // dz
                    x[i][e] = d * gate;
                } else {
                    x[i][e] = d;
                }
            }
        store<T, TPU, VPT, VEC>((T *)p.dx + row * a.channels + c0, x, th, D);
        if (gated || pre) store<T, TPU, VPT, VEC>((T *)p.dz + row * a.channels + c0, z, th, D);
    }
    if (p.pw && first < p.splits) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = chan<TPU, VEC>(th, i, e);
                if (c < D) {
                    p.pw[first * a.channels + c0 + c] = dw[i][e];
                    p.pb[first * a.channels + c0 + c] = db[i][e];
                }
            }
    }
}

// dweight, dbias = sums of the shares, in a fixed order: 8 rows of threads
// each add every 8th share, then one row adds the 8 sums.
__global__ void __launch_bounds__(256) norm_shares_kernel(const float *pw, const float *pb, int splits, int64_t C, float *dw, float *db) {
    __shared__ float sm[8][32][2];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x % 32;
    const int y = threadIdx.x / 32;
    float u = 0.f, v = 0.f;
    if (c < C)
        for (int s = y; s < splits; s += 8) {
            u += pw[(int64_t)s * C + c];
            v += pb[(int64_t)s * C + c];
        }
    sm[y][threadIdx.x % 32][0] = u;
    sm[y][threadIdx.x % 32][1] = v;
    __syncthreads();
    if (y == 0 && c < C) {
        u = v = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u += sm[i][threadIdx.x][0];
            v += sm[i][threadIdx.x][1];
        }
        if (dw) dw[c] = u;
        if (db) db[c] = v;
    }
}

// Threads per unit and 8-channel vectors per thread for a group of D channels:
// the narrowest unit that holds the group, so that few lanes idle.
struct Shape {
    int tpu, vpt;
};
Shape shape_of(int64_t D) {
    if (D <= 64) return {8, 1};
    if (D <= 128) return {16, 1};
    if (D <= 256) return {32, 1};
    if (D <= 512) return {32, 2};
    if (D <= 1024) return {128, 1};
    if (D <= 2048) return {128, 2};
    if (D <= 4096) return {256, 2};
    return {512, 4};
}

int splits_of(const ssm_norm_args &a, int ctas_per_sm) {
    const Shape s = shape_of(a.channels / a.groups);
    const int threads = s.tpu > 256 ? s.tpu : 256, upb = threads / s.tpu;
    const int64_t rows = a.batch * a.seqlen;
    const int64_t units = (int64_t)sm_count() * ctas_per_sm * upb;
    int64_t n = units / a.groups;
    if (n < 1) n = 1;
    return (int)(n < rows ? n : rows);
}
// CTAs per SM: as many as the registers allow (two 512-thread CTAs at most).
int fwd_ctas(const ssm_norm_args &a) { return shape_of(a.channels / a.groups).tpu > 256 ? 1 : 4; }
int bwd_ctas(const ssm_norm_args &a) { return shape_of(a.channels / a.groups).tpu > 256 ? 1 : 2; }

template <bool BWD, typename T, int TPU, int VPT>
void run(const Args &p, bool vec, cudaStream_t st) {
    constexpr int UPB = threads_of<TPU>() / TPU;
    const int64_t units = (int64_t)p.splits * p.a.groups;
    const unsigned grid = (unsigned)((units + UPB - 1) / UPB);
    if constexpr (BWD) {
        if (vec) group_norm_bwd_kernel<T, TPU, VPT, true><<<grid, threads_of<TPU>(), 0, st>>>(p);
        else group_norm_bwd_kernel<T, TPU, VPT, false><<<grid, threads_of<TPU>(), 0, st>>>(p);
    } else {
        if (vec) group_norm_kernel<T, TPU, VPT, true><<<grid, threads_of<TPU>(), 0, st>>>(p);
        else group_norm_kernel<T, TPU, VPT, false><<<grid, threads_of<TPU>(), 0, st>>>(p);
    }
}
template <bool BWD, typename T>
cudaError_t pick(const Args &p, bool vec, cudaStream_t st) {
    const Shape s = shape_of(p.a.channels / p.a.groups);
    timing_begin(st);
    if (s.tpu == 8) run<BWD, T, 8, 1>(p, vec, st);
    else if (s.tpu == 16) run<BWD, T, 16, 1>(p, vec, st);
    else if (s.tpu == 32 && s.vpt == 1) run<BWD, T, 32, 1>(p, vec, st);
    else if (s.tpu == 32) run<BWD, T, 32, 2>(p, vec, st);
    else if (s.tpu == 128 && s.vpt == 1) run<BWD, T, 128, 1>(p, vec, st);
    else if (s.tpu == 128) run<BWD, T, 128, 2>(p, vec, st);
    else if (s.tpu == 256) run<BWD, T, 256, 2>(p, vec, st);
    else run<BWD, T, 512, 4>(p, vec, st);
    timing_end(st);
    return cudaGetLastError();
}

// 16-byte accesses need groups of whole 8-channel runs and aligned rows.
bool vec_ok(const void *p, int64_t bs, int64_t ts, size_t es) {
    return !p || ((uintptr_t)p % 16 == 0 && bs * (int64_t)es % 16 == 0 && ts * (int64_t)es % 16 == 0);
}

}  // namespace

cudaError_t launch_group_norm(const ssm_norm_args &a, cudaStream_t st) {
    Args p{};
    p.a = a;
    p.rows = a.batch * a.seqlen;
    if (p.rows == 0) return cudaSuccess;
    p.splits = splits_of(a, fwd_ctas(a));
    const size_t es = a.dtype == SSM_BF16 ? 2 : 4;
    const bool vec = (a.channels / a.groups) % 8 == 0 && vec_ok(a.x, a.x_batch_stride, a.x_token_stride, es) &&
                     vec_ok(a.z, a.z_batch_stride, a.z_token_stride, es) &&
                     vec_ok(a.y, a.y_batch_stride, a.y_token_stride, es);
    return a.dtype == SSM_BF16 ? pick<false, __nv_bfloat16>(p, vec, st) : pick<false, float>(p, vec, st);
}

size_t group_norm_bwd_workspace_bytes(const ssm_norm_bwd_args &b) {
    const ssm_norm_args &a = b.fwd;
    if (a.batch * a.seqlen == 0) return 0;
    return 2 * (((size_t)splits_of(a, bwd_ctas(a)) * a.channels * 4 + 255) / 256 * 256);
}

cudaError_t launch_group_norm_bwd(const ssm_norm_bwd_args &b, void *ws, cudaStream_t st) {
    const ssm_norm_args &a = b.fwd;
    Args p{};
    p.a = a;
    p.dy = b.dy;
    p.dy_bs = b.dy_batch_stride;
    p.dy_ts = b.dy_token_stride;
    p.dx = b.dx;
    p.dz = b.dz;
    p.rows = a.batch * a.seqlen;
    if (p.rows == 0) {
        cudaError_t e = cudaSuccess;
        if (b.dweight) e = cudaMemsetAsync(b.dweight, 0, a.channels * 4, st);
        if (e == cudaSuccess && b.dbias) e = cudaMemsetAsync(b.dbias, 0, a.channels * 4, st);
        return e;
    }
    p.splits = splits_of(a, bwd_ctas(a));
    if (b.dweight || b.dbias) {
        p.pw = static_cast<float *>(ws);
        p.pb = reinterpret_cast<float *>(static_cast<char *>(ws) + group_norm_bwd_workspace_bytes(b) / 2);
    }
    const size_t es = a.dtype == SSM_BF16 ? 2 : 4;
    const bool vec = (a.channels / a.groups) % 8 == 0 && vec_ok(a.x, a.x_batch_stride, a.x_token_stride, es) &&
                     vec_ok(a.z, a.z_batch_stride, a.z_token_stride, es) &&
                     vec_ok(b.dy, b.dy_batch_stride, b.dy_token_stride, es) && vec_ok(b.dx, 0, 0, es) &&
                     vec_ok(b.dz, 0, 0, es);
    cudaError_t e = a.dtype == SSM_BF16 ? pick<true, __nv_bfloat16>(p, vec, st) : pick<true, float>(p, vec, st);
    if (e != cudaSuccess || !p.pw) return e;
    norm_shares_kernel<<<(unsigned)((a.channels + 31) / 32), 256, 0, st>>>(p.pw, p.pb, p.splits, a.channels, b.dweight,
                                                                          b.dbias);
    return cudaGetLastError();
}

}  // namespace ssm
