// group_norm.cu -- group norm of channels-last rows with an activation or a
// SiLU gate, forward and backward (formulas in ssm.h).
//
// A unit of TPU threads owns one group of every `stride`-th token and keeps
// the group in registers between the statistics and the output, so x (and z)
// are read once and y is written once: HBM-bound.  Units next to each other in
// a CTA own the groups next to each other of one token, so a CTA reads a
// contiguous stretch.  A unit stays with its group, which keeps the weights
// (forward) and their gradients' sums (backward) in registers over its tokens.
// Groups of 512, gate behind the norm: 402 MB in 75 us, 5.4 TB/s; groups of 64
// with the gate in front, backward: 671 MB in 141 us, 4.8 TB/s.  Units of 512
// threads have 128 registers a thread and spill: the backward from 4097 channels
// a group on (up to 620 bytes a thread, past 8192 channels 1 to 2 KB), the
// forward past 8192 with fp32 or a gate (60 to 390 bytes).
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
    int64_t share;           // values that each share array has room for
};

// Sum of u (and of v) over the unit's TPU threads; every thread gets it.
// `red` holds 2 floats per warp of the CTA.
template <int TPU, bool TWO>
SSM_DEVINL void unit_sum(float &u, float &v, float *red) {
#pragma unroll
    for (int o = 1; o < (TPU < 32 ? TPU : 32); o <<= 1) {
        u += __shfl_xor_sync(~0u, u, o);
        if (TWO) v += __shfl_xor_sync(~0u, v, o);
    }
    if constexpr (TPU > 32) {
        const int warp = threadIdx.x >> 5, first = warp / (TPU / 32) * (TPU / 32);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
            red[2 * warp] = u;
            if (TWO) red[2 * warp + 1] = v;
        }
        __syncthreads();
        u = v = 0.f;
#pragma unroll
        for (int i = 0; i < TPU / 32; ++i) {
            u += red[2 * (first + i)];
            if (TWO) v += red[2 * (first + i) + 1];
        }
    }
}

// Channel (within the group) of value e of vector i of this thread: runs of 8
// (16-byte accesses), or one channel per thread and step.
template <int TPU, bool VEC>
SSM_DEVINL int chan(int th, int i, int e) {
    return VEC ? (i * TPU + th) * 8 + e : (i * 8 + e) * TPU + th;
}
// Whether the group holds it (VEC: groups are whole runs, so e does not matter).
template <int TPU, bool VEC>
SSM_DEVINL bool held(int th, int i, int e, int D) { return chan<TPU, VEC>(th, i, VEC ? 0 : e) < D; }

// 8 VPT values of this thread as they lie in memory: bf16 stays packed until it
// is used, which halves the registers that loads in flight occupy.
template <typename T, int VPT> struct Raw;
template <int VPT> struct Raw<float, VPT> {
    float v[VPT][8];
    SSM_DEVINL float get(int i, int e) const { return v[i][e]; }
};
template <int VPT> struct Raw<__nv_bfloat16, VPT> {
    uint32_t w[VPT][4];
    SSM_DEVINL float get(int i, int e) const {
        return __uint_as_float(e & 1 ? w[i][e >> 1] & 0xffff0000u : w[i][e >> 1] << 16);
    }
};
template <typename T, int TPU, int VPT, bool VEC>
SSM_DEVINL void load(Raw<T, VPT> &r, const T *p, int th, int D) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (VEC && sizeof(T) == 2) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (held<TPU, VEC>(th, i, 0, D)) x = *reinterpret_cast<const uint4 *>(p + chan<TPU, VEC>(th, i, 0));
            r.w[i][0] = x.x; r.w[i][1] = x.y; r.w[i][2] = x.z; r.w[i][3] = x.w;
        } else if constexpr (VEC) {
            if (held<TPU, VEC>(th, i, 0, D)) Vec8<float>::ld(p + chan<TPU, VEC>(th, i, 0), r.v[i]);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) r.v[i][e] = 0.f;
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const int c0 = chan<TPU, VEC>(th, i, e), c1 = chan<TPU, VEC>(th, i, e + 1);
                const uint32_t x = c0 < D ? __bfloat16_as_ushort(p[c0]) : 0, y = c1 < D ? __bfloat16_as_ushort(p[c1]) : 0;
                r.w[i][e >> 1] = x | y << 16;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = chan<TPU, VEC>(th, i, e);
                r.v[i][e] = c < D ? p[c] : 0.f;
            }
        }
    }
}
template <typename T, int TPU, int VPT, bool VEC>
SSM_DEVINL void store(T *p, const float (&v)[8], int th, int i, int D) {
    if constexpr (VEC) {
        if (held<TPU, VEC>(th, i, 0, D)) Vec8<T>::st(p + chan<TPU, VEC>(th, i, 0), v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = chan<TPU, VEC>(th, i, e);
            if (c < D) Elem<T>::st(p + c, v[e]);
        }
    }
}

// 1 / (1 + e^-v) on the MUFU unit: two operations of 2^-22 relative error each;
// for v << 0 the power overflows to infinity and its reciprocal is 0.
SSM_DEVINL float sigmoid(float v) { return rcp(1.f + ex2(-v * kLog2e)); }

// Batch and token of a row number (rows < 2^31): no division for one batch row.
SSM_DEVINL void split_row(const ssm_norm_args &a, int64_t row, int64_t &b, int64_t &t) {
    b = 0;
    t = row;
    if (a.batch > 1) {
        const uint32_t n = (uint32_t)a.seqlen, q = (uint32_t)row / n;
        b = q;
        t = (uint32_t)row - q * n;
    }
}

// Whether the row and its channels up to c lie in the tensors (the bounds-checked build; else true).
SSM_DEVINL bool in_tensor(const ssm_norm_args &a, int64_t b, int64_t t, int64_t c) {
    return SSM_BOUNDS(b, a.batch, BS_NORM_ROW) && SSM_BOUNDS(t, a.seqlen, BS_NORM_ROW) &&
           SSM_BOUNDS(c, a.channels, BS_NORM_CHANNEL);
}

template <int TPU> constexpr int threads_of() { return TPU > 256 ? TPU : 256; }
// What z does: nothing, gate the result, gate the input.
enum Kind { kNoGate, kGate, kGateFirst };

// mean and 1 / sqrt(var + eps) of the group whose values this unit's threads
// give (zeros past the group): the mean first, then the centred squares, which
// loses no digits however far the mean is from zero.
template <int TPU, int VPT, bool VEC, typename F>
SSM_DEVINL void stats(F get, int th, int D, float inv, bool centre, float eps, float *red, float &mean, float &r) {
    float m2 = 0.f, none = 0.f;
    mean = 0.f;
    if (centre) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) mean += get(i, e);
        unit_sum<TPU, false>(mean, none, red);
        mean *= inv;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = held<TPU, VEC>(th, i, e, D) ? get(i, e) - mean : 0.f;
            m2 = fmaf(d, d, m2);
        }
    unit_sum<TPU, false>(m2, none, red);
    r = rsqrtf(fmaf(m2, inv, eps));
}

template <typename T, int TPU, int VPT, bool VEC, Kind K>
__global__ void __launch_bounds__(threads_of<TPU>()) group_norm_kernel(const Args p) {
    __shared__ float red[threads_of<TPU>() / 32 * 2];
    const ssm_norm_args &a = p.a;
    constexpr int UPB = threads_of<TPU>() / TPU;
    const int th = threadIdx.x % TPU, D = (int)(a.channels / a.groups);
    const float inv = 1.f / (float)D;
    const int64_t unit = (int64_t)blockIdx.x * UPB + threadIdx.x / TPU;
    const int64_t grp = unit % a.groups, first = unit / a.groups;
    const int64_t c0 = grp * D;
    const bool act = a.mode == SSM_NORM_SILU;
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
    const int turns = (int)((p.rows + p.splits - 1) / p.splits);
    Raw<T, VPT> x, z;
    const auto fetch = [&](int it, Raw<T, VPT> &x, Raw<T, VPT> &z) {
        const int64_t row = first + (int64_t)it * p.splits;
        const bool live = first < p.splits && row < p.rows;
        int64_t bi, t;
        split_row(a, live ? row : 0, bi, t);
        const int dl = live && in_tensor(a, bi, t, c0 + D - 1) ? D : 0;
        load<T, TPU, VPT, VEC>(x, (const T *)a.x + bi * a.x_batch_stride + t * a.x_token_stride + c0, th, dl);
        if (K != kNoGate)
            load<T, TPU, VPT, VEC>(z, (const T *)a.z + bi * a.z_batch_stride + t * a.z_token_stride + c0, th, dl);
    };
    fetch(0, x, z);
    for (int it = 0; it < turns; ++it) {
        const int64_t row = first + (int64_t)it * p.splits;
        const bool live = first < p.splits && row < p.rows;
        if (TPU <= 32 && __all_sync(~0u, !live)) break;
        Raw<T, VPT> xn, zn;                            // the next token's values, in flight meanwhile
        if (it + 1 < turns) fetch(it + 1, xn, zn);
        float s[K == kGateFirst ? VPT : 1][8];
        if (K == kGateFirst)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) s[K == kGateFirst ? i : 0][e] = x.get(i, e) * z.get(i, e) * sigmoid(z.get(i, e));
        const auto in = [&](int i, int e) { return K == kGateFirst ? s[K == kGateFirst ? i : 0][e] : x.get(i, e); };
        float mean, r;
        stats<TPU, VPT, VEC>(in, th, D, inv, a.subtract_mean != 0, a.eps, red, mean, r);
        if (live) {
            int64_t bi, t;
            split_row(a, row, bi, t);
            const int ds = in_tensor(a, bi, t, c0 + D - 1) ? D : 0;
            T *y = (T *)a.y + bi * a.y_batch_stride + t * a.y_token_stride + c0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float v = fmaf((in(i, e) - mean) * r, w[i][e], b[i][e]);
                    if (K == kGate) v *= z.get(i, e) * sigmoid(z.get(i, e));
                    if (K == kNoGate && act) v *= sigmoid(v);
                    o[e] = v;
                }
                store<T, TPU, VPT, VEC>(y, o, th, i, ds);
            }
        }
        x = xn;
        z = zn;
    }
}

// (one vector per thread: two CTAs an SM and at most 128 registers; more vectors: all that a thread can have)
template <typename T, int TPU, int VPT, bool VEC, Kind K>
__global__ void __launch_bounds__(threads_of<TPU>(), VPT == 1 ? 2 : 1) group_norm_bwd_kernel(const Args p) {
    __shared__ float red[threads_of<TPU>() / 32 * 2];
    const ssm_norm_args &a = p.a;
    constexpr int UPB = threads_of<TPU>() / TPU;
    const int th = threadIdx.x % TPU, D = (int)(a.channels / a.groups);
    const int64_t unit = (int64_t)blockIdx.x * UPB + threadIdx.x / TPU;
    const int64_t grp = unit % a.groups, first = unit / a.groups;
    const int64_t c0 = grp * D;
    const bool act = a.mode == SSM_NORM_SILU;
    const float inv = 1.f / (float)D;
    float w[VPT][8], b[VPT][8], dw[VPT][8], db[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = chan<TPU, VEC>(th, i, e);
            w[i][e] = a.weight && c < D ? a.weight[c0 + c] : 1.f;
            // the bias matters only where the gradient looks at t itself
            b[i][e] = K != kGateFirst && a.bias && c < D ? a.bias[c0 + c] : 0.f;
            dw[i][e] = db[i][e] = 0.f;
        }
    const int turns = (int)((p.rows + p.splits - 1) / p.splits);
    Raw<T, VPT> x, z, g;
    const auto fetch = [&](int it, Raw<T, VPT> &x, Raw<T, VPT> &z, Raw<T, VPT> &g) {
        const int64_t row = first + (int64_t)it * p.splits;
        const bool live = first < p.splits && row < p.rows;
        int64_t bi, t;
        split_row(a, live ? row : 0, bi, t);
        const int dl = live && in_tensor(a, bi, t, c0 + D - 1) ? D : 0;
        load<T, TPU, VPT, VEC>(x, (const T *)a.x + bi * a.x_batch_stride + t * a.x_token_stride + c0, th, dl);
        load<T, TPU, VPT, VEC>(g, (const T *)p.dy + bi * p.dy_bs + t * p.dy_ts + c0, th, dl);
        if (K != kNoGate)
            load<T, TPU, VPT, VEC>(z, (const T *)a.z + bi * a.z_batch_stride + t * a.z_token_stride + c0, th, dl);
    };
    fetch(0, x, z, g);
    for (int it = 0; it < turns; ++it) {
        const int64_t row = first + (int64_t)it * p.splits;
        const bool live = first < p.splits && row < p.rows;
        if (TPU <= 32 && __all_sync(~0u, !live)) break;
        Raw<T, VPT> xn, zn, gn;
        // with up to two vectors per thread there are registers for the next token's loads
        if (VPT <= 2 && it + 1 < turns) fetch(it + 1, xn, zn, gn);
        float s[VPT][8], sg[K == kNoGate ? 1 : VPT][8], dn[VPT][8];
        float dz[K == kGate ? VPT : 1][8];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (K != kNoGate) sg[K == kNoGate ? 0 : i][e] = sigmoid(z.get(i, e));
                s[i][e] = K == kGateFirst ? x.get(i, e) * (z.get(i, e) * sg[K == kNoGate ? 0 : i][e]) : x.get(i, e);
            }
        float mean, r;
        stats<TPU, VPT, VEC>([&](int i, int e) { return s[i][e]; }, th, D, inv, a.subtract_mean != 0, a.eps, red, mean, r);
        if (!live) r = 0.f;                            // (eps = 0: 1 / sqrt(0) of no token must not meet dy = 0)
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // dy is 0 past the group and for a token that is not there, and with it all that is summed
                const float n = (s[i][e] - mean) * r;
                float dt = g.get(i, e);
                if (K == kGate) {
                    const float sv = sg[K == kNoGate ? 0 : i][e], gate = z.get(i, e) * sv;
                    dz[K == kGate ? i : 0][e] = dt * fmaf(n, w[i][e], b[i][e]) * fmaf(gate, 1.f - sv, sv);
                    dt *= gate;
                } else if (K == kNoGate && act) {
                    const float t = fmaf(n, w[i][e], b[i][e]), sv = sigmoid(t);
                    dt *= fmaf(t * sv, 1.f - sv, sv);
                }
                s[i][e] = n;
                dw[i][e] = fmaf(dt, n, dw[i][e]);
                db[i][e] += dt;
                dn[i][e] = dt * w[i][e];
                s1 += dn[i][e];
                s2 = fmaf(dn[i][e], n, s2);
            }
        unit_sum<TPU, true>(s1, s2, red);
        if (live) {
            s1 = a.subtract_mean ? s1 * inv : 0.f;
            s2 *= inv;
            const int ds = SSM_BOUNDS(row * a.channels + c0 + D - 1, p.rows * a.channels, BS_NORM_ROW) ? D : 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float o[8], o2[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float d = r * (dn[i][e] - s1 - s[i][e] * s2);
                    o[e] = d;
                    if (K == kGateFirst) {
                        const float sv = sg[K == kNoGate ? 0 : i][e], gate = z.get(i, e) * sv;
                        o2[e] = d * x.get(i, e) * fmaf(gate, 1.f - sv, sv);
                        o[e] = d * gate;
                    } else if (K == kGate) {
                        o2[e] = dz[K == kGate ? i : 0][e];
                    }
                }
                store<T, TPU, VPT, VEC>((T *)p.dx + row * a.channels + c0, o, th, i, ds);
                if (K != kNoGate) store<T, TPU, VPT, VEC>((T *)p.dz + row * a.channels + c0, o2, th, i, ds);
            }
        }
        if (VPT <= 2) {
            x = xn;
            z = zn;
            g = gn;
        } else if (it + 1 < turns) {
            fetch(it + 1, x, z, g);
        }
    }
    if (p.pw && first < p.splits) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = chan<TPU, VEC>(th, i, e);
                if (c < D && SSM_BOUNDS(first * a.channels + c0 + c, p.share, BS_NORM_SHARE)) {
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
// the narrowest unit that holds the group, so that few lanes idle; in the backward,
// which holds four times as much, and without 16-byte accesses in single vectors
// where those do not cost a wider unit.  Gated
// forward / backward of 16384 rows of 4096 bf16 channels in us, and with another
// shape: D 64 79 / 133 (units of 32 threads 295 / 468), D 128 77 / 134 (153 / 243),
// D 512 74 / 140 (64 threads of one vector 81 / 151, 128 threads 125 / 267), D 2048
// 79 / 155 (forward as the backward 83, backward as the forward 179), D 4096
// 79 / 160 (512 threads of one vector 90 / 173); rows of one group of 8192: 159 / 490
// (four vectors 342 / 1637).  Without 16-byte accesses D 63 132 / 218 (32 threads
// 374 / 645), D 511 140 / 225 (128 threads 249 / 404), D 2047 117 / 234 (two vectors
// 268 / 596).
struct Shape {
    int tpu, vpt;
};
Shape shape_of(int64_t D, bool vec, bool bwd) {
    if (D <= 64) return {8, 1};
    if (D <= 128) return {16, 1};
    if (D <= 256) return {32, 1};
    if (D <= 512) return vec ? Shape{32, 2} : Shape{64, 1};
    if (D <= 1024) return {128, 1};
    if (D <= 2048) return vec && !bwd ? Shape{128, 2} : Shape{256, 1};
    if (D <= 4096) return {256, 2};
    return D <= 8192 ? Shape{512, 2} : Shape{512, 4};
}

// Units per group: as many as fill the GPU at so many warps per SM, so that a
// unit keeps its weights over many tokens.
constexpr int kFwdWarps = 32, kBwdWarps = 16;
int splits_of(const ssm_norm_args &a, bool vec, bool bwd) {
    const Shape s = shape_of(a.channels / a.groups, vec, bwd);
    const int64_t rows = a.batch * a.seqlen, units = (int64_t)sm_count() * (bwd ? kBwdWarps : kFwdWarps) * 32 / s.tpu;
    int64_t n = units / a.groups;
    if (n < 1) n = 1;
    return (int)(n < rows ? n : rows);
}

template <bool BWD, typename T, int TPU, int VPT, bool VEC, Kind K>
void run(const Args &p, cudaStream_t st) {
    constexpr int UPB = threads_of<TPU>() / TPU;
    const int64_t units = (int64_t)p.splits * p.a.groups;
    const unsigned grid = (unsigned)((units + UPB - 1) / UPB);
    if constexpr (BWD) group_norm_bwd_kernel<T, TPU, VPT, VEC, K><<<grid, threads_of<TPU>(), 0, st>>>(p);
    else group_norm_kernel<T, TPU, VPT, VEC, K><<<grid, threads_of<TPU>(), 0, st>>>(p);
}
template <bool BWD, typename T, bool VEC, Kind K>
void with(const Args &p, Shape s, cudaStream_t st) {
    if (s.tpu == 8) run<BWD, T, 8, 1, VEC, K>(p, st);
    else if (s.tpu == 16) run<BWD, T, 16, 1, VEC, K>(p, st);
    else if (s.tpu == 32 && s.vpt == 1) run<BWD, T, 32, 1, VEC, K>(p, st);
    else if (s.tpu == 128 && s.vpt == 1) run<BWD, T, 128, 1, VEC, K>(p, st);
    else if (s.tpu == 32 || s.tpu == 64) run<BWD, T, VEC ? 32 : 64, VEC ? 2 : 1, VEC, K>(p, st);
    else if (s.tpu == 128 || (s.tpu == 256 && s.vpt == 1))
        run<BWD, T, VEC && !BWD ? 128 : 256, VEC && !BWD ? 2 : 1, VEC, K>(p, st);
    else if (s.tpu == 256) run<BWD, T, 256, 2, VEC, K>(p, st);
    else if (s.vpt == 2) run<BWD, T, 512, 2, VEC, K>(p, st);
    else run<BWD, T, 512, 4, VEC, K>(p, st);
}
template <bool BWD, typename T, Kind K>
void pick(const Args &p, bool vec, cudaStream_t st) {
    const Shape s = shape_of(p.a.channels / p.a.groups, vec, BWD);
    if (vec) with<BWD, T, true, K>(p, s, st);
    else with<BWD, T, false, K>(p, s, st);
}
template <bool BWD>
cudaError_t launch(const Args &p, bool vec, cudaStream_t st) {
    const bool bf = p.a.dtype == SSM_BF16;
    timing_begin(st);
    if (p.a.mode == SSM_NORM_GATE) bf ? pick<BWD, __nv_bfloat16, kGate>(p, vec, st) : pick<BWD, float, kGate>(p, vec, st);
    else if (p.a.mode == SSM_NORM_GATE_FIRST)
        bf ? pick<BWD, __nv_bfloat16, kGateFirst>(p, vec, st) : pick<BWD, float, kGateFirst>(p, vec, st);
    else bf ? pick<BWD, __nv_bfloat16, kNoGate>(p, vec, st) : pick<BWD, float, kNoGate>(p, vec, st);
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
    const size_t es = a.dtype == SSM_BF16 ? 2 : 4;
    const bool vec = (a.channels / a.groups) % 8 == 0 && vec_ok(a.x, a.x_batch_stride, a.x_token_stride, es) &&
                     vec_ok(a.z, a.z_batch_stride, a.z_token_stride, es) &&
                     vec_ok(a.y, a.y_batch_stride, a.y_token_stride, es);
    p.splits = splits_of(a, vec, false);
    return launch<false>(p, vec, st);
}

size_t group_norm_bwd_workspace_bytes(const ssm_norm_bwd_args &b) {
    const ssm_norm_args &a = b.fwd;
    if (a.batch * a.seqlen == 0) return 0;
    // shapes alone decide the size: room for the layout with more units per group
    const int n = splits_of(a, true, true), m = splits_of(a, false, true);
    return 2 * (((size_t)(n > m ? n : m) * a.channels * 4 + 255) / 256 * 256);
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
    if (b.dweight || b.dbias) {
        p.pw = static_cast<float *>(ws);
        const size_t half = group_norm_bwd_workspace_bytes(b) / 2;
        p.pb = reinterpret_cast<float *>(static_cast<char *>(ws) + half);
        p.share = (int64_t)(half / 4);
    }
    const size_t es = a.dtype == SSM_BF16 ? 2 : 4;
    const bool vec = (a.channels / a.groups) % 8 == 0 && vec_ok(a.x, a.x_batch_stride, a.x_token_stride, es) &&
                     vec_ok(a.z, a.z_batch_stride, a.z_token_stride, es) &&
                     vec_ok(b.dy, b.dy_batch_stride, b.dy_token_stride, es) && vec_ok(b.dx, 0, 0, es) &&
                     vec_ok(b.dz, 0, 0, es);
    p.splits = splits_of(a, vec, true);
    cudaError_t e = launch<true>(p, vec, st);
    if (e != cudaSuccess || !p.pw) return e;
    norm_shares_kernel<<<(unsigned)((a.channels + 31) / 32), 256, 0, st>>>(p.pw, p.pb, p.splits, a.channels, b.dweight,
                                                                          b.dbias);
    return cudaGetLastError();
}

}  // namespace ssm
