// delta_tc_bwd.cu -- backward of the blocked gated delta rule on the tensor
// cores (bf16 activations, dstate <= 128).  Per block of 64 tokens, with h the
// entering state, d = dL/d(leaving state), P the attention weights (scale in
// them), T, R, U as in the forward, e_ij = exp(cs_i - cs_j):
//
//   dU = P^T dy + diag(exp(cs_last - cs)) K d^T,     dR = T^T dU,
//   dv = beta dR,                 dS = -beta exp(cs) dR  (gradient of h k),
//   d <- exp(cs_last) d + sum_i scale exp(cs_i) dy_i q_i^T + sum_j dS_j k_j^T;
//   A_ij = scale e_ij (dy_i . u_j) (j <= i),  B_ij = -beta_i e_ij (dR_i . u_j) (j < i),
//   dq = scale exp(cs) dy h + A K,
//   dk = dS h + exp(cs_last - cs) u d + A^T Q + (B + B^T) K,
//   dbeta_i = dR_i . u_i / beta_i,
//   dg_t = sum_{i >= t} (dq_i . q_i - dk_i . k_i + 2 dR_i . (u_i - beta_i v_i)) + <h_out, d>.
//
// The line of dg: every factor exp(cs_i - cs_j) weighs a product of q_i or k_i
// on the side of i and of k_j on that of j, so the sums over a row or a column
// are dot products of the finished gradients with q and k, and no second pass
// over the 64 x 64 matrices is needed; u - beta v = -beta (exp(cs) h k + sum e (k.k) u).
//
// Three launches after the pre-pass: the states' pass (delta_tc_fwd.cu) from
// the first block to the last, the gradients' chain here from the last to the
// first, which leaves dv, dh0 and its operands, and one CTA per (block, group)
// that makes dq, dk, dg and dbeta of all the group's heads, so that dq and dk
// are summed in a fixed order and rounded once.
//
// dg_t is a difference: terms of two tokens behind t stand in dq . q, in dk . k
// and in dR . (u - beta v) and cancel.  All of them use the same rounded matrix,
// so what is left of them is the rounding of fp32 sums: 5e-6 where the block's
// terms are about 1, whatever a_t is.  Every other term holds a_t itself.
//
// Rounding: on the way to dh0 every factor that is not exact goes as two bf16
// parts (as in the forward), and so does all of dv but its own rounding (1.7e-3
// of its norm).  The last launch takes h, d, dR, u and the matrices A and B as
// single bf16 values: dq and dk are off by 2.9e-3 of their norm, dbeta by 2.3e-3,
// where rounding the exact values gives 1.7e-3.  Second parts would make a
// slice's record 104 KB instead of 56, and a CTA holds two: more than an SM's
// shared memory, for gradients that are bf16 when they leave.
//
// 4 x 2048 tokens, 16 heads of P 128 in 8 groups, N 128: pre-pass 52 us, states'
// pass 111, gradients' chain 150 (both chains' latency: 64 CTAs, 32 blocks each),
// the blocks' gradients 124 (230 MB of kept operands; one CTA an SM, whose
// products, passes and loads follow one another, 14k cycles a head).
#include <string.h>

#include "delta_tc.cuh"
#include "delta_tc.h"

namespace ssm {
namespace {

using namespace dtc;

// ============================================================ gradients' chain
constexpr int kChainWarps = 8, kSideWarps = 4;
constexpr int kSide0 = kChainWarps, kMmaWarp = kSide0 + kSideWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = (kLoadWarp + 1) * 32;
static_assert(kSide0 % 4 == 0, "lane quarters");
// tensor-memory columns
constexpr uint32_t TM_D = 0;       // fp32 gradient of the state, decayed for the next block
constexpr uint32_t TM_DOP = 128;   // its two bf16 parts (as TM_HOP of the forward); then scale exp(cs) dy, two parts
constexpr uint32_t TM_X1 = 256;    // d k, then dR (two heads: in 128 columns)
constexpr uint32_t TM_X2 = 320;    // dy^T P
constexpr uint32_t TM_OP = 384;    // dU, then dS: two parts of 32 columns
constexpr uint32_t TM_DY = 448;    // dy as an operand (exact)
constexpr uint32_t kTmemCols = 512;

enum Bar {
    B_FULL0, B_FULL1, B_EMPTY0, B_EMPTY1, B_TAB0, B_TAB1, B_PFULL, B_PEMPTY,
    B_D0, B_D1, B_X1, B_DU0, B_DU1, B_DR, B_DS0, B_DS1, B_NEXT,      // the chain
    B_DY, B_X2, B_DYQ, B_RREAD,                                      // beside it
    B_DRAIN, B_COUNT
};

SSM_DEVINL uint32_t dop(int cf, int b, int part) { return TM_DOP + 64 * b + 32 * part + 16 * cf; }

struct alignas(16) Tab {
    float beta[kQ], bg[kQ], w[kQ], gs[kQ];
    float total;
};
struct Aux {
    uint64_t mb[B_COUNT];
    uint32_t tmem;
    int abort;
    Tab tab[2][2];
};

template <int NK, bool DUAL> struct Lay {
    static constexpr uint32_t kKB = NK / 64 * 2 * kTile;
    static constexpr uint32_t kTPart = (DUAL ? 2 : 1) * kTile;
    static constexpr uint32_t K = 0, DY = kKB, T = DY + 2 * kTile, stage = T + 2 * kTPart;
    static constexpr uint32_t P = 2 * stage, V = P + 2 * kTPart, AUX = V + 2 * kTile;    // P: one buffer
    static constexpr size_t bytes = AUX + sizeof(Aux) + 1024;
};

struct Args {
    ssm_delta_bwd_args b;
    SeqView sv;
    const uint8_t *prep;
    Rec rec;
    int64_t nblk, slots;
    int R, nsl, units;
};

template <int NK, bool DUAL>
__global__ void __launch_bounds__(kThreads, 1)
delta_bwd_chain_kernel(const Args p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_dy) {
    using L = Lay<NK, DUAL>;
    const ssm_delta_args &a = p.b.fwd;
    if (p.sv.err && *p.sv.err != 0) return;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = smem_1024(raw);
    Aux &ax = *reinterpret_cast<Aux *>(sm + L::AUX);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int grp = blockIdx.x / p.units, unit = blockIdx.x % p.units;
    const int half0 = 2 * unit, halves = min(2, p.R * p.nsl - half0);
    int head[2], row0[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int hf = half0 + min(i, halves - 1);
        head[i] = grp * p.R + hf / p.nsl;
        row0[i] = hf % p.nsl * 64;
    }
    int s;
    int64_t brow, lo, hi;
    if (a.cu_seqlens) {
        s = p.sv.order[blockIdx.y];
        brow = 0;
        lo = a.cu_seqlens[s];
        hi = a.cu_seqlens[s + 1];
    } else {
        s = blockIdx.y;
        brow = s;
        lo = 0;
        hi = a.seqlen;
    }
    if (!SSM_BOUNDS(hi, a.seqlen + 1, BS_DELTA_SEQ) || !SSM_BOUNDS(lo, hi + 1, BS_DELTA_SEQ)) return;
    const int n = (int)((hi - lo + kQ - 1) / kQ);
    const int64_t H = a.nheads, P = a.headdim, N = a.dstate;
    if (n == 0) {
        if (p.b.dh0)
            for (int i = 0; i < halves; ++i)
                for (int64_t e = tid; e < min((int64_t)64, P - row0[i]) * N; e += kThreads) {
                    const int64_t at = (((int64_t)s * H + head[i]) * P + row0[i]) * N + e;
                    p.b.dh0[at] = p.b.dh_final ? p.b.dh_final[at] : 0.f;
                }
        return;
    }
    const int64_t slot0 = seq_slot(a.cu_seqlens, s, p.nblk);
    if (!SSM_BOUNDS(slot0 + n - 1, p.slots, BS_DELTA_SLOT) || !SSM_BOUNDS(max(head[0], head[1]), H, BS_DELTA_HEAD) ||
        !SSM_BOUNDS(max(row0[0], row0[1]), P, BS_DELTA_STATE)) return;
    if (warp == 0) tc::tmem_alloc(&ax.tmem, kTmemCols);
    if (tid == 0) {
        constexpr int kEmpty = 1 + kChainWarps + kSideWarps;
        constexpr int counts[B_COUNT] = {
            1, 1, kEmpty, kEmpty, 1, 1, 1, 1,
            kChainWarps, kChainWarps, 1, kChainWarps, kChainWarps, 1, kChainWarps, kChainWarps, 1,
            kSideWarps, 1, kSideWarps, kSideWarps,
            1};
        for (int i = 0; i < B_COUNT; ++i) tc::mbar_init(&ax.mb[i], counts[i]);
        tc::mbar_init_fence();
        ax.abort = 0;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = ax.tmem;
    volatile int *ab = &ax.abort;
    int32_t *err = p.sv.err;
    auto wait = [&](int b, uint32_t parity) { return wait_warp(&ax.mb[b], ab, parity, err); };
    const uint32_t sb = tc::smem_u32(sm);
    int issued = 0;                            // turns whose loads the load warp has issued
    // blocks run from the last: turn `it` is block n - 1 - it
    auto tokens = [&](int it) { return (int)min((int64_t)kQ, hi - lo - (int64_t)(n - 1 - it) * kQ); };

    if (warp < kChainWarps) {
        const int q = warp & 3, cf = warp >> 2, half = q >> 1, rr = (q & 1) * 32 + lane, r = row0[half] + rr;
        const bool live = half < halves && r < P;
        const uint32_t tl = tm + ((uint32_t)(32 * q) << 16);
        const int64_t srow = (((int64_t)s * H + head[half]) * P + r) * N;
        auto arrive_st = [&](int b) {
            tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive(&ax.mb[b]);
        };
        // 32 columns of the gradient that leaves block c
        auto keep = [&](int c, int col, const float *v) {
            if (half >= halves) return;
            uint8_t *rec = p.rec.at(slot0 + c, H, head[half], row0[half] / 64) + p.rec.state;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint4 o = make_uint4(0, 0, 0, 0);
                const float *f = v + 8 * k;
                if (live) o = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
                *reinterpret_cast<uint4 *>(rec + rec_off(rr, col + 8 * k)) = o;
            }
        };
        bool ok = wait(B_TAB0, 0);
        float x[32], h1[32];
        uint32_t raw_[32], raw1[32];
#pragma unroll
        for (int b = 0; b < NK / 64; ++b) {
            const int c0 = cf * (NK / 2) + b * 32;
            float *v = b ? h1 : x;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (live && p.b.dh_final && c0 + i < N) f = *reinterpret_cast<const float4 *>(p.b.dh_final + srow + c0 + i);
                v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
            }
        }
        float total = ax.tab[0][half].total;
        for (int it = 0; it <= n && ok; ++it) {
            // x, h1: the gradient that leaves block n - 1 - it (it = n: that of h0)
            if (it == n) {
                if (p.b.dh0 && live)
#pragma unroll
                    for (int b = 0; b < NK / 64; ++b)
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const int c0 = cf * (NK / 2) + b * 32 + i;
                            const float *f = (b ? h1 : x) + i;
                            if (c0 < N)
                                *reinterpret_cast<float4 *>(p.b.dh0 + srow + c0) = make_float4(f[0], f[1], f[2], f[3]);
                        }
                break;
            }
#pragma unroll
            for (int b = 0; b < NK / 64; ++b) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    st_split16(tl + dop(cf, b, 0) + 8 * e, tl + dop(cf, b, 1) + 8 * e, (b ? h1 : x) + 16 * e);
                arrive_st(B_D0 + b);
            }
            if (NK == 64 && lane == 0) arrive(&ax.mb[B_D1]);
            // decayed for this block's update; dU, handed over later, covers these stores
#pragma unroll
            for (int b = 0; b < NK / 64; ++b) {
                keep(n - 1 - it, cf * (NK / 2) + b * 32, b ? h1 : x);
                float *f = b ? h1 : x;
#pragma unroll
                for (int i = 0; i < 32; ++i) f[i] *= total;
                tmem_st32(tl + TM_D + cf * (NK / 2) + b * 32, b ? h1 : x);
            }
            const uint32_t ph = it & 1;
            const int stg = it & 1, nt = tokens(it), t0 = cf * 32;
            uint8_t *st = sm + stg * L::stage;
            const Tab &tb = ax.tab[stg][half];
            // dU = dy^T P + exp(cs_last - cs) d k
            {
                float w[32];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 w4 = *reinterpret_cast<const float4 *>(tb.w + t0 + i);
                    w[i] = w4.x; w[i + 1] = w4.y; w[i + 2] = w4.z; w[i + 3] = w4.w;
                }
                ok = wait(B_FULL0 + stg, (it >> 1) & 1) && wait(B_X2, ph) && wait(B_X1, ph);
                if (!ok) break;
                tc::fence_after_sync();
                tmem_ld32_start(tl + TM_X1 + t0, raw_);
                tmem_ld32_start(tl + TM_X2 + t0, raw1);
                if (nt < kQ) {                 // keys and queries behind the sequence's end may be anything
                    for (int i = tid; i < 2 * (kQ - nt) * (NK / 8); i += kChainWarps * 32) {
                        const int k = i % (NK / 8) * 8, z = i / (NK / 8), row = nt + (z >> 1);
                        *reinterpret_cast<uint4 *>(st + L::K + (k >> 6) * 2 * kTile + (z & 1) * kTile + swz(row, k & 63)) =
                            make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_proxy_async();
                }
                float y[32];
                tmem_ld32_wait(raw_, x);
                tmem_ld32_wait(raw1, y);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = t0 + i < nt ? fmaf(w[i], x[i], y[i]) : 0.f;
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                st_split16(tl + TM_OP + t0 / 2 + 8 * b, tl + TM_OP + 32 + t0 / 2 + 8 * b, x + 16 * b);
                arrive_st(B_DU0 + b);
            }
            // dS = -beta exp(cs) dR
            {
                float bg[32];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 g4 = *reinterpret_cast<const float4 *>(tb.bg + t0 + i);
                    bg[i] = g4.x; bg[i + 1] = g4.y; bg[i + 2] = g4.z; bg[i + 3] = g4.w;
                }
                ok = wait(B_DR, ph);
                if (!ok) break;
                tc::fence_after_sync();
                tmem_ld32_start(tl + TM_X1 + (DUAL && half ? 64 : 0) + t0, raw_);
                tmem_ld32_wait(raw_, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] *= -bg[i];
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                st_split16(tl + TM_OP + t0 / 2 + 8 * b, tl + TM_OP + 32 + t0 / 2 + 8 * b, x + 16 * b);
                arrive_st(B_DS0 + b);
            }
            if (lane == 0) arrive(&ax.mb[B_EMPTY0 + stg]);
            // d
            if (it + 1 < n) {
                ok = wait(B_TAB0 + (stg ^ 1), ((it + 1) >> 1) & 1);
                if (!ok) break;
                total = ax.tab[stg ^ 1][half].total;
            }
            ok = wait(B_NEXT, ph);
            if (!ok) break;
            tc::fence_after_sync();
            tmem_ld32_start(tl + TM_D + cf * (NK / 2), raw_);
            if (NK == 128) tmem_ld32_start(tl + TM_D + cf * (NK / 2) + 32, raw1);
            tmem_ld32_wait(raw_, x);
            if (NK == 128) tmem_ld32_wait(raw1, h1);
        }
    } else if (warp < kMmaWarp) {
        // ------------------------------------------- dy as operands; dv, dR out
        const int q = warp - kSide0, half = q >> 1, rr = (q & 1) * 32 + lane;
        const bool live = half < halves && row0[half] + rr < P;
        const uint32_t tl = tm + ((uint32_t)(32 * q) << 16);
        const int ch = (32 * q + lane) & 15, vh = ch >> 3;
        const bool in = vh < halves && row0[vh] + (ch & 7) * 8 < P;
        __nv_bfloat16 *dv = static_cast<__nv_bfloat16 *>(p.b.dv) + ((brow * a.seqlen + lo) * H + head[vh]) * P + row0[vh] +
                            (ch & 7) * 8;
        __nv_bfloat16 *vs = reinterpret_cast<__nv_bfloat16 *>(sm + L::V);
        uint32_t dy[32];                           // this row's dy, two tokens each
        auto arrive_w = [&](int b) {
            __syncwarp();
            if (lane == 0) arrive(&ax.mb[b]);
        };
        // dy of turn `it` into tensor memory and, transposed, into the records
        auto take_dy = [&](int it) {
            const int stg = it & 1, nt = tokens(it);
            if (!wait(B_FULL0 + stg, (it >> 1) & 1)) return false;
            const uint16_t *v = reinterpret_cast<const uint16_t *>(sm + stg * L::stage + L::DY + half * kTile) + rr;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const uint32_t x = live && 2 * i < nt ? v[2 * i * 64] : 0, y = live && 2 * i + 1 < nt ? v[(2 * i + 1) * 64] : 0;
                dy[i] = x | y << 16;
            }
            if (it > 0 && !wait(B_X2, (it - 1) & 1)) return false;
            uint32_t h[16];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int i = 0; i < 16; ++i) h[i] = dy[16 * b + i];
                tmem_st16(tl + TM_DY + 16 * b, h);
            }
            tmem_wait_st();
            tc::fence_before_sync();
            arrive_w(B_DY);
            if (half < halves) {
                uint8_t *rec = p.rec.at(slot0 + n - 1 - it, H, head[half], row0[half] / 64) + p.rec.dy();
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<uint4 *>(rec + rec_off(rr, 8 * k)) =
                        make_uint4(dy[4 * k], dy[4 * k + 1], dy[4 * k + 2], dy[4 * k + 3]);
            }
            return true;
        };
        bool ok = take_dy(0);
        for (int it = 0; it < n; ++it) {
            const uint32_t ph = it & 1;
            const int stg = it & 1, nt = tokens(it);
            const Tab &tb = ax.tab[stg][half];
            // scale exp(cs) dy over d's operand, which the product with k has used
            ok = ok && wait(B_TAB0 + stg, (it >> 1) & 1) && wait(B_X1, ph);
            tc::fence_after_sync();
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float f[16];
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 g = *reinterpret_cast<const float4 *>(tb.gs + 16 * b + i);
                    const uint32_t u = dy[8 * b + i / 2], v = dy[8 * b + i / 2 + 1];
                    f[i] = g.x * __uint_as_float(u << 16);
                    f[i + 1] = g.y * __uint_as_float(u & 0xffff0000u);
                    f[i + 2] = g.z * __uint_as_float(v << 16);
                    f[i + 3] = g.w * __uint_as_float(v & 0xffff0000u);
                }
                st_split16(tl + TM_DOP + 8 * b, tl + TM_DOP + 32 + 8 * b, f);
            }
            tmem_wait_st();
            tc::fence_before_sync();
            arrive_w(B_DYQ);
            if (it + 1 < n) ok = ok && take_dy(it + 1);
            // dR: dv = beta dR by way of shared memory, and dR itself for the last launch
            ok = ok && wait(B_DR, ph);
            tc::fence_after_sync();
            float x[2][32];
            uint32_t r0[32], r1[32];
            tmem_ld32_start(tl + TM_X1 + (DUAL && half ? 64 : 0), r0);
            tmem_ld32_start(tl + TM_X1 + (DUAL && half ? 64 : 0) + 32, r1);
            tmem_ld32_wait(r0, x[0]);
            tmem_ld32_wait(r1, x[1]);
            tc::fence_before_sync();
            arrive_w(B_RREAD);
            uint8_t *rec = p.rec.at(slot0 + n - 1 - it, H, head[half], row0[half] / 64) + p.rec.dR();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float *f = x[b];
                if (half < halves && ok)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint4 o = make_uint4(0, 0, 0, 0);
                        if (live)
                            o = make_uint4(pack2(f[8 * k], f[8 * k + 1]), pack2(f[8 * k + 2], f[8 * k + 3]),
                                           pack2(f[8 * k + 4], f[8 * k + 5]), pack2(f[8 * k + 6], f[8 * k + 7]));
                        *reinterpret_cast<uint4 *>(rec + rec_off(rr, 32 * b + 8 * k)) = o;
                    }
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 be = *reinterpret_cast<const float4 *>(tb.beta + 32 * b + i);
                    __nv_bfloat16 *at = vs + (32 * b + i) * 128 + 32 * q + lane;
                    at[0] = __float2bfloat16_rn(be.x * f[i]);
                    at[128] = __float2bfloat16_rn(be.y * f[i + 1]);
                    at[256] = __float2bfloat16_rn(be.z * f[i + 2]);
                    at[384] = __float2bfloat16_rn(be.w * f[i + 3]);
                }
            }
            if (lane == 0) arrive(&ax.mb[B_EMPTY0 + stg]);
            if (!bar_all<128>(ok)) break;
            if (in) {
                __nv_bfloat16 *o = dv + (int64_t)(n - 1 - it) * kQ * H * P;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = 2 * q + (lane >> 4) + 8 * i;
                    if (t < nt && SSM_BOUNDS(lo + (int64_t)(n - 1 - it) * kQ + t, a.seqlen, BS_DELTA_OUT))
                        *reinterpret_cast<uint4 *>(o + (int64_t)t * H * P) = *reinterpret_cast<const uint4 *>(vs + t * 128 + ch * 8);
                }
            }
            asm volatile("bar.sync 1, 128;\n" ::: "memory");
        }
    } else if (warp == kMmaWarp) {
        constexpr uint32_t ID1 = tc::idesc_bf16(128, 64, 0, 0), IDT = tc::idesc_bf16(128, DUAL ? 128 : 64, 0, 1),
                           IDP = tc::idesc_bf16(128, 64, 0, 1), IDN = tc::idesc_bf16(128, NK, 0, 1);
        // dy^T P of a turn
        auto x2 = [&](int it) {
            const uint32_t ph = it & 1;
            if (!wait(B_PFULL, ph) || !wait(B_DY, ph) || (it > 0 && !wait(B_RREAD, ph ^ 1))) return false;
            tc::fence_after_sync();
            if (lane == 0) {
#pragma unroll 1
                for (int hh = 0; hh < (DUAL ? 2 : 1); ++hh) {
                    const uint64_t dP = tc::desc_sw128(sb + L::P + hh * kTile, kTile, 1024);
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint64_t B = dP + (part ? 0 : L::kTPart >> 4) + kk * 128;
                            if constexpr (DUAL)
                                mma_ts_lanes(tm + TM_X2, tm + TM_DY + kk * 8, B, IDP, part + kk > 0, hh ? ~0u : 0u,
                                             hh ? 0u : ~0u);
                            else
                                mma_ts(tm + TM_X2, tm + TM_DY + kk * 8, B, IDP, part + kk > 0);
                        }
                }
                tc::mma_commit(&ax.mb[B_X2]);
                tc::mma_commit(&ax.mb[B_PEMPTY]);
            }
            __syncwarp();
            return true;
        };
        bool ok = x2(0);
        for (int it = 0; it < n && ok; ++it) {
            const uint32_t ph = it & 1;
            const int stg = it & 1;
            const uint32_t st = sb + stg * L::stage;
            const uint64_t dK = tc::desc_sw128(st + L::K, 16, 1024), dKm = tc::desc_sw128(st + L::K, 2 * kTile, 1024);
            const uint64_t dT = tc::desc_sw128(st + L::T, kTile, 1024);
            // d k, over the last dR (read)
            ok = wait(B_FULL0 + stg, (it >> 1) & 1) && (it == 0 || wait(B_RREAD, ph ^ 1));
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                ok = ok && wait(B_D0 + b, ph);
                if (!ok) break;
                tc::fence_after_sync();
                if (lane == 0) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k4 = 0; k4 < NK / 32; ++k4) {
                            const int kk = NK == 64 ? 2 * b + k4 : (k4 >> 1) * 4 + 2 * b + (k4 & 1);
                            mma_ts(tm + TM_X1, tm + dop(NK == 64 ? b : k4 >> 1, NK == 64 ? 0 : b, part) + (k4 & 1) * 8,
                                   dK + (((kk >> 2) * 2 * kTile + (kk & 3) * 32) >> 4), ID1, b + part + k4 > 0);
                        }
                    if (b) tc::mma_commit(&ax.mb[B_X1]);
                }
                __syncwarp();
            }
            // dR = T^T dU: (dU high, T low), (dU low, T high), (dU high, T high)
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                ok = ok && wait(B_DU0 + b, ph);
                if (!ok) break;
                tc::fence_after_sync();
                if (lane == 0) {
#pragma unroll
                    for (int part = 0; part < 3; ++part)
#pragma unroll
                        for (int k2 = 0, kk = b; k2 < 2; ++k2, kk += 2)
                            mma_ts(tm + TM_X1, tm + TM_OP + (part == 1 ? 32 : 0) + kk * 8,
                                   dT + (part == 0 ? L::kTPart >> 4 : 0) + kk * 128, IDT, b + part + kk > 0);
                    if (b) tc::mma_commit(&ax.mb[B_DR]);
                }
                __syncwarp();
            }
            // the state's gradient: scale exp(cs) dy q while dS is made, then dS k
            ok = ok && wait(B_DYQ, ph);
            if (!ok) break;
            tc::fence_after_sync();
            if (lane == 0)
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ts(tm + TM_D, tm + TM_DOP + part * 32 + kk * 8, dKm + (kTile >> 4) + kk * 128, IDN, 1);
            __syncwarp();
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                ok = ok && wait(B_DS0 + b, ph);
                if (!ok) break;
                tc::fence_after_sync();
                if (lane == 0) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k2 = 0, kk = b; k2 < 2; ++k2, kk += 2)
                            mma_ts(tm + TM_D, tm + TM_OP + part * 32 + kk * 8, dKm + kk * 128, IDN, 1);
                    if (b) {
                        tc::mma_commit(&ax.mb[B_NEXT]);
                        tc::mma_commit(&ax.mb[B_EMPTY0 + stg]);
                    }
                }
                __syncwarp();
            }
            if (ok && it + 1 < n) ok = x2(it + 1);
        }
    } else {
        // --------------------------------------------------- loads and gate tables
        for (int it = 0; it < n; ++it) {
            const int stg = it & 1, blk = n - 1 - it, nt = tokens(it);
            const int64_t t0 = lo + (int64_t)blk * kQ;
            float gv[2][2], bv[2][2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = lane + 32 * e;
                    const bool in = t < nt && (hh == 0 || head[1] != head[0]);
                    gv[hh][e] = in ? a.g[brow * a.g_batch_stride + (t0 + t) * a.g_token_stride + head[hh]] : 0.f;
                    bv[hh][e] = bwd_beta(in ? a.beta[brow * a.beta_batch_stride + (t0 + t) * a.beta_token_stride + head[hh]] : 0.f);
                }
            if (it >= 2 && !wait(B_EMPTY0 + stg, ((it >> 1) - 1) & 1)) break;
            if (it >= 1 && !wait(B_PEMPTY, (it - 1) & 1)) break;
            uint8_t *st = sm + stg * L::stage;
            if (lane == 0) {
                uint64_t *mb = &ax.mb[B_FULL0 + stg];
                tc::mbar_expect_tx(&ax.mb[B_PFULL], 2 * L::kTPart);
                tc::mbar_expect_tx(mb, L::stage);
#pragma unroll
                for (int i = 0; i < (DUAL ? 2 : 1); ++i) {
                    const uint8_t *src = p.prep + ((slot0 + blk) * H + head[i]) * kHeadBytesBwd;
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        bulk_load(sm + L::P + part * L::kTPart + i * kTile, src + (2 + part) * kTile, kTile, &ax.mb[B_PFULL]);
                        bulk_load(st + L::T + part * L::kTPart + i * kTile, src + part * kTile, kTile, mb);
                    }
                }
#pragma unroll
                for (int x = 0; x < NK / 64; ++x) {
                    tma_load_4d(st + L::K + x * 2 * kTile, &tm_k, 64 * x, grp, (int)t0, (int)brow, mb);
                    tma_load_4d(st + L::K + x * 2 * kTile + kTile, &tm_q, 64 * x, grp, (int)t0, (int)brow, mb);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    tc::tma_load_3d(st + L::DY + i * kTile, &tm_dy, (int)(head[i] * P + row0[i]), (int)t0, (int)brow, mb);
            }
            issued = it + 1;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                Tab &tb = ax.tab[stg][hh];
                if (hh == 1 && head[1] == head[0]) {
                    gv[1][0] = gv[0][0]; gv[1][1] = gv[0][1];
                    bv[1][0] = bv[0][0]; bv[1][1] = bv[0][1];
                }
                double cs[2], last;
                block_cs(log_decay(gv[hh][0]), log_decay(gv[hh][1]), cs[0], cs[1], last);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = lane + 32 * e;
                    const float ec = exp_d(cs[e]);
                    tb.beta[t] = bv[hh][e];
                    tb.bg[t] = bv[hh][e] * ec;
                    tb.w[t] = exp_d(last - cs[e]);
                    tb.gs[t] = a.scale * ec;
                }
                if (lane == 0) tb.total = exp_d(last);
            }
            __syncwarp();
            if (lane == 0) arrive(&ax.mb[B_TAB0 + stg]);
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (*ab) {                                 // (as in the forward chain)
        if (warp < kMmaWarp) tmem_wait_st();
        if (warp == kLoadWarp && lane == 0 && issued > 0) {
            for (int c = max(0, issued - 2); c < issued; ++c) tc::mbar_wait(&ax.mb[B_FULL0 + (c & 1)], (c >> 1) & 1, 1u << 22);
            tc::mbar_wait(&ax.mb[B_PFULL], (issued - 1) & 1, 1u << 22);
        }
        if (warp == kMmaWarp && lane == 0) {
            tc::mma_commit(&ax.mb[B_DRAIN]);
            tc::mbar_wait(&ax.mb[B_DRAIN], 0, 1u << 22);
        }
        __syncwarp();
        tc::fence_before_sync();
        __syncthreads();
    }
    if (warp == 0) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tm, kTmemCols);
    }
}

// ================================================= dq, dk, dg, dbeta of a block
constexpr int kGradThreads = 256;
// tensor-memory columns: [dy; dR] u^T, [dy; dR] h, u d (upper lanes), the attention part; K K^T (upper lanes)
constexpr uint32_t TG_U = 0, TG_H = 64, TG_D = 192, TG_A = 320, TG_K = 448;

struct GradArgs {
    ssm_delta_bwd_args b;
    SeqView sv;
    Rec rec;
    int64_t nblk;
    int R, nsl;
};
// (cs in one part: after 64 resets it is 1e4, where its rounding moves a weight by 2^-11; the weight is then rounded
// to bf16, up to 2^-8)
struct alignas(16) GradTab {
    float cs[kQ], beta[kQ], bg[kQ], w[kQ], gs[kQ];
    float total;
};
struct GradAux {
    uint64_t full, done;
    uint32_t tmem;
    int abort;
    GradTab tab;
    float dot[2][2 * kQ];          // per column half: dq . q of row i, dk . k of row 64 + i
    float zw[2][kQ], ew[2][kQ];    // dR . (u - beta v), exp(cs_last - cs) (u d) . k
    float ru[kQ];                  // dR . u
    float hd[kGradThreads / 32];
};
template <int NK> struct GradLay {
    static constexpr uint32_t kAtoms = NK / 64;
    static constexpr uint32_t QK = 0;                                  // per 64 states: Q rows, K rows
    static constexpr uint32_t A = kAtoms * 2 * kTile;                  // 128 x 128: two 64-column atoms of 128 rows
    static constexpr uint32_t REC = A + 4 * kTile;                     // two slices: h, d, dy, dR, u
    static constexpr uint32_t rec = (2 * kAtoms + 3) * kTile;
    static constexpr uint32_t AUX = REC + 2 * rec;
    static constexpr size_t bytes = AUX + sizeof(GradAux) + 1024;
};

template <int NK>
__global__ void __launch_bounds__(kGradThreads, 1)
delta_grad_kernel(const GradArgs p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k) {
    using L = GradLay<NK>;
    const ssm_delta_args &a = p.b.fwd;
    if (p.sv.err && *p.sv.err != 0) return;
    const Block blk = find_block(a.cu_seqlens, p.sv.nseqs, a.seqlen, p.nblk, blockIdx.x);
    if (blk.nt == 0) return;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = smem_1024(raw);
    GradAux &ax = *reinterpret_cast<GradAux *>(sm + L::AUX);
    const uint32_t sb = tc::smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = blockIdx.y;
    const int quarter = warp & 3, cf = warp >> 2, r = 32 * quarter + lane, i = r & 63;    // row; token
    const bool upper = r >= 64;                                                          // a dk row
    const int64_t H = a.nheads, N = a.dstate;
    const int nt = blk.nt;
    if (!SSM_BOUNDS(blk.s, p.sv.nseqs, BS_DELTA_SEQ) || !SSM_BOUNDS(blk.t0 + nt - 1, a.seqlen, BS_DELTA_OUT) ||
        !SSM_BOUNDS(grp * p.R + p.R - 1, H, BS_DELTA_HEAD)) return;
    if (warp == 0) tc::tmem_alloc(&ax.tmem, 512);
    if (tid == 0) {
        tc::mbar_init(&ax.full, 1);
        tc::mbar_init(&ax.done, 1);
        tc::mbar_init_fence();
        ax.abort = 0;
    }
    // dq has no part over Q: those columns of its rows stay zero
    for (int x = tid; x < 64 * 8; x += kGradThreads)
        *reinterpret_cast<uint4 *>(sm + L::A + x * 16) = make_uint4(0, 0, 0, 0);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = ax.tmem, tl = tm + ((uint32_t)(32 * quarter) << 16);
    uint32_t nfull = 0, ndone = 0, loads = 0, products = 0;    // phases waited for; (thread 0) started
    bool ok = true;
    auto full = [&] { ok = wait_bar(&ax.full, &ax.abort, nfull++ & 1, p.sv.err) && ok; };
    auto done = [&] {
        ok = wait_bar(&ax.done, &ax.abort, ndone++ & 1, p.sv.err) && ok;
        tc::fence_after_sync();
    };
    // slices s0, s0 + 1 of a head's records
    auto load = [&](int head, int s0) {
        const int ns = min(2, p.nsl - s0);
        ++loads;
        tc::mbar_expect_tx(&ax.full, ns * L::rec);
        for (int x = 0; x < ns; ++x)
            bulk_load(sm + L::REC + x * L::rec, p.rec.at(blockIdx.x, H, head, s0 + x), L::rec, &ax.full);
    };
    if (tid == 0) {
        ++loads;
        tc::mbar_expect_tx(&ax.full, L::A);
#pragma unroll
        for (int x = 0; x < NK / 64; ++x) {
            tma_load_4d(sm + L::QK + x * 2 * kTile, &tm_q, 64 * x, grp, (int)blk.t0, (int)blk.row, &ax.full);
            tma_load_4d(sm + L::QK + x * 2 * kTile + kTile, &tm_k, 64 * x, grp, (int)blk.t0, (int)blk.row, &ax.full);
        }
    }
    full();
    if (nt < kQ) {                             // queries and keys behind the sequence's end may be anything
        for (int x = tid; x < 2 * (kQ - nt) * (NK / 8); x += kGradThreads) {
            const int k = x % (NK / 8) * 8, z = x / (NK / 8), row = nt + (z >> 1);
            *reinterpret_cast<uint4 *>(sm + L::QK + (k >> 6) * 2 * kTile + (z & 1) * kTile + swz(row, k & 63)) =
                make_uint4(0, 0, 0, 0);
        }
    }
    tc::fence_proxy_async();
    if (!__syncthreads_and(ok)) ok = false;
    const uint64_t dQK = tc::desc_sw128(sb + L::QK, 16, 1024), dQKm = tc::desc_sw128(sb + L::QK, 2 * kTile, 1024);
    if (ok && tid == 0) {
        load(grp * p.R, 0);
#pragma unroll 1
        for (int kk = 0; kk < NK / 16; ++kk) {
            const uint32_t o = ((kk >> 2) * 2 * kTile + (kk & 3) * 32) >> 4;
            tc::mma_bf16(tm + TG_K, dQK + o, dQK + (kTile >> 4) + o, tc::idesc_bf16(128, 64, 0, 0), kk > 0);
        }
        tc::mma_commit(&ax.done);
        ++products;
    }
    __syncwarp();
    if (ok) done();
    float acc[NK / 2];
#pragma unroll
    for (int e = 0; e < NK / 2; ++e) acc[e] = 0.f;
    const uint8_t *own = sm + L::QK + (upper ? kTile : 0);             // this row's q or k

    for (int hh = 0; hh < p.R; ++hh) {
        const int head = grp * p.R + hh;
        float keep[2];                                 // warp 0: 0 at a reset, whose dg = a <d, h> is exactly zero
        if (warp == 0) {
            const float *gp = a.g + blk.row * a.g_batch_stride + blk.t0 * a.g_token_stride + head;
            const float *bp = a.beta + blk.row * a.beta_batch_stride + blk.t0 * a.beta_token_stride + head;
            double cs[2], last;
            const float g0 = lane < nt ? log_decay(gp[lane * a.g_token_stride]) : 0.f;
            const float g1 = lane + 32 < nt ? log_decay(gp[(lane + 32) * a.g_token_stride]) : 0.f;
            keep[0] = resets(g0) ? 0.f : 1.f;
            keep[1] = resets(g1) ? 0.f : 1.f;
            block_cs(g0, g1, cs[0], cs[1], last);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = lane + 32 * e;
                const float be = bwd_beta(t < nt ? bp[t * a.beta_token_stride] : 0.f), ec = exp_d(cs[e]);
                ax.tab.cs[t] = (float)(cs[e] * 1.4426950408889634);
                ax.tab.beta[t] = be;
                ax.tab.bg[t] = be * ec;
                ax.tab.w[t] = exp_d(last - cs[e]);
                ax.tab.gs[t] = a.scale * ec;
            }
            if (lane == 0) ax.tab.total = exp_d(last);
        }
        // the products over the head's rows, two 64-row slices at a time; <h, d> beside them
        float hd = 0.f;
        for (int s0 = 0; s0 < p.nsl; s0 += 2) {
            const int ns = min(2, p.nsl - s0);
            if (ok) full();
            if (!__syncthreads_and(ok)) {
                ok = false;
                break;
            }
            if (tid == 0) {
                tc::fence_after_sync();
                for (int x = 0; x < ns; ++x) {
                    const uint32_t rec = sb + L::REC + x * L::rec;
                    const uint64_t dH = tc::desc(rec, 128, 1024), dD = dH + (L::kAtoms * kTile >> 4);
                    const uint64_t dY = dD + (L::kAtoms * kTile >> 4), dR = dY + (kTile >> 4), dU = dR + (kTile >> 4);
#pragma unroll 1
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t o = kk * 16, c = s0 + x + kk > 0;
                        tc::mma_bf16(tm + TG_U, dY + o, dU + o, tc::idesc_bf16(128, 64, 1, 1), c);
                        tc::mma_bf16(tm + TG_H, dY + o, dH + o, tc::idesc_bf16(128, NK, 1, 1), c);
                        tc::mma_bf16(tm + TG_D, dR + o, dD + o, tc::idesc_bf16(128, NK, 1, 1), c);
                    }
                }
                tc::mma_commit(&ax.done);
                ++products;
            }
            __syncwarp();
            for (int x = 0; x < ns; ++x) {
                constexpr int kPer = L::kAtoms * kTile / 16 / kGradThreads;
                uint4 hv[kPer], dv[kPer];
#pragma unroll
                for (int y = 0; y < kPer; ++y) {
                    const uint8_t *t = sm + L::REC + x * L::rec + (tid + y * kGradThreads) * 16;
                    hv[y] = *reinterpret_cast<const uint4 *>(t);
                    dv[y] = *reinterpret_cast<const uint4 *>(t + L::kAtoms * kTile);
                }
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int y = 0; y < kPer; ++y) {
                    float u[8], v[8];
                    tc::unpack_bf16x8(hv[y], u);
                    tc::unpack_bf16x8(dv[y], v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) part[e & 3] = fmaf(u[e], v[e], part[e & 3]);
                }
                hd += (part[0] + part[1]) + (part[2] + part[3]);
            }
            done();
            if (!__syncthreads_and(ok)) {              // the tiles are read and used
                ok = false;
                break;
            }
            if (tid == 0) {
                if (s0 + 2 < p.nsl) load(head, s0 + 2);
                else if (hh + 1 < p.R) load(head + 1, 0);
            }
        }
        if (!ok) break;
#pragma unroll
        for (int o = 16; o; o >>= 1) hd += __shfl_xor_sync(~0u, hd, o);
        if (lane == 0) ax.hd[warp] = hd;
        // the 128 x 128 matrix over [Q; K]: rows of dq [0 | A], rows of dk [A^T | B + B^T]
        float x[32], zw = 0.f;
        {
            const int j0 = 32 * cf;
            const float ci = ax.tab.cs[i], f = upper ? -ax.tab.beta[i] : a.scale;
            float cj[32], own_x = 0.f;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4 c4 = *reinterpret_cast<const float4 *>(ax.tab.cs + j0 + e);
                cj[e] = c4.x; cj[e + 1] = c4.y; cj[e + 2] = c4.z; cj[e + 3] = c4.w;
            }
            tc::tmem_ld32(tl + TG_U + j0, x);
            const int last = i < nt ? (upper ? i - 1 : i) - j0 : -1;   // columns up to it count
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                if (e == i - j0) own_x = x[e];
                x[e] = e <= last ? f * ex2(ci - cj[e]) * x[e] : 0.f;
            }
            if (upper && (unsigned)(i - j0) < 32u) ax.ru[i] = own_x;
            // from here on x is the rounded value that the matrix holds: in dg the pairs of two tokens behind t come
            // from dk . k (twice) and from zw, and cancel only if all three are the same number
            uint8_t *row = sm + L::A + 2 * kTile;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float *v = x + 8 * k + 2 * e;
                    o[e] = pack2(v[0], v[1]);
                    v[0] = __uint_as_float(o[e] << 16);
                    v[1] = __uint_as_float(o[e] & 0xffff0000u);
                }
                *reinterpret_cast<uint4 *>(row + swz(r, j0 + 8 * k)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            if (upper) {
                float kk[32];
                tc::tmem_ld32(tl + TG_K + j0, kk);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (j0 + e < i) zw = fmaf(x[e], kk[e], zw);
            }
            __syncthreads();                           // the rows are written: the transposed parts go over their zeros
            uint8_t *col = sm + L::A + (upper ? 2 * kTile : 0);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const int j = j0 + e;
                if (!upper || j < i)
                    *reinterpret_cast<__nv_bfloat16 *>(col + swz(64 + j, i)) = __float2bfloat16_rn(x[e]);
            }
        }
        tc::fence_proxy_async();
        tc::fence_before_sync();
        __syncthreads();
        if (tid == 0) {
            tc::fence_after_sync();
            const uint64_t dA = tc::desc_sw128(sb + L::A, 16, 1024);
#pragma unroll 1
            for (int kk = 0; kk < 8; ++kk)
                tc::mma_bf16(tm + TG_A, dA + (((kk >> 2) * 2 * kTile + (kk & 3) * 32) >> 4), dQKm + kk * 128,
                             tc::idesc_bf16(128, NK, 0, 1), kk > 0);
            tc::mma_commit(&ax.done);
            ++products;
        }
        __syncwarp();
        done();
        // the gradients of this head's q and k rows, and their dot products with the rows
        {
            const float fh = upper ? -ax.tab.bg[i] : ax.tab.gs[i], fd = ax.tab.w[i];
            float dot = 0.f, ew = 0.f;
#pragma unroll
            for (int b = 0; b < NK / 64; ++b) {
                const int c0 = cf * (NK / 2) + 32 * b;
                float y[32], z[32];
                tc::tmem_ld32(tl + TG_H + c0, y);
                tc::tmem_ld32(tl + TG_A + c0, z);
                if (upper) tc::tmem_ld32(tl + TG_D + c0, x);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float o[8];
                    const int c = c0 + 8 * k;
                    tc::unpack_bf16x8(*reinterpret_cast<const uint4 *>(own + (c >> 6) * 2 * kTile + swz(i, c & 63)), o);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float vh = fh * y[8 * k + e], vd = upper ? fd * x[8 * k + e] : 0.f;
                        const float v = vh + z[8 * k + e] + vd;
                        acc[32 * b + 8 * k + e] += v;
                        dot = fmaf(v, o[e], dot);
                        if (upper) {
                            zw = fmaf(vh, o[e], zw);
                            ew = fmaf(vd, o[e], ew);
                        }
                    }
                }
            }
            ax.dot[cf][r] = dot;
            if (upper) {
                ax.zw[cf][i] = zw;
                ax.ew[cf][i] = ew;
            }
        }
        tc::fence_before_sync();
        __syncthreads();
        if (warp == 0) {
            float d[2], e = 0.f, last = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = lane + 32 * h;
                const bool in = t < nt;
                d[h] = in ? ax.dot[0][t] + ax.dot[1][t] - ax.dot[0][64 + t] - ax.dot[1][64 + t] +
                                2.f * (ax.zw[0][t] + ax.zw[1][t]) : 0.f;
                e += in ? ax.ew[0][t] + ax.ew[1][t] : 0.f;
            }
#pragma unroll
            for (int w = 0; w < kGradThreads / 32; ++w) last += ax.hd[w];
#pragma unroll
            for (int o = 16; o; o >>= 1) e += __shfl_xor_sync(~0u, e, o);
            last = fmaf(ax.tab.total, last, e);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {         // sums over the tokens from t on
                const float u = __shfl_down_sync(~0u, d[0], o), v = __shfl_down_sync(~0u, d[1], o);
                if (lane + o < 32) {
                    d[0] += u;
                    d[1] += v;
                }
            }
            d[0] += __shfl_sync(~0u, d[1], 0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = lane + 32 * h;
                if (t < nt) {
                    const int64_t at = (blk.row * a.seqlen + blk.t0 + t) * H + head;
                    store_gates<__nv_bfloat16>(p.b, at, keep[h] * (d[h] + last), ax.ru[t] / ax.tab.beta[t]);
                }
            }
        }
        __syncthreads();
    }
    // dq and dk by way of the matrix's place: a lane's own row would take a line per store.  16-byte pieces, those of
    // neighbouring rows in different banks.
    if (__syncthreads_and(ok)) {
        constexpr int kRow = NK / 8;
#pragma unroll
        for (int k = 0; k < NK / 16; ++k)
            *reinterpret_cast<uint4 *>(sm + L::A + (r * kRow + ((cf * (NK / 16) + k) ^ (r & 7))) * 16) =
                make_uint4(pack2(acc[8 * k], acc[8 * k + 1]), pack2(acc[8 * k + 2], acc[8 * k + 3]),
                           pack2(acc[8 * k + 4], acc[8 * k + 5]), pack2(acc[8 * k + 6], acc[8 * k + 7]));
        __syncthreads();
#pragma unroll
        for (int y = 0; y < 128 * kRow / kGradThreads; ++y) {
            const int x = tid + y * kGradThreads, row = x / kRow, c = x % kRow;
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(row >= 64 ? p.b.dk : p.b.dq) +
                               ((blk.row * a.seqlen + blk.t0 + (row & 63)) * a.ngroups + grp) * N + c * 8;
            if ((row & 63) < nt && c * 8 < N)
                *reinterpret_cast<uint4 *>(o) =
                    *reinterpret_cast<const uint4 *>(sm + L::A + (row * kRow + (c ^ (row & 7))) * 16);
        }
    }
    if (ax.abort && tid == 0) {
        // a wait ran out: what is in flight (the last phase started of each barrier) lands before the CTA ends
        if (products) tc::mbar_wait(&ax.done, (products - 1) & 1, 1u << 22);
        if (loads) tc::mbar_wait(&ax.full, (loads - 1) & 1, 1u << 22);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tm, 512);
    }
}

template <int NK, bool DUAL>
cudaError_t run_chain(const Args &p, dim3 grid, const DeltaMaps &m, const CUtensorMap &dy, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(delta_bwd_chain_kernel<NK, DUAL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Lay<NK, DUAL>::bytes);
    if (e != cudaSuccess) return e;
    delta_bwd_chain_kernel<NK, DUAL><<<grid, kThreads, Lay<NK, DUAL>::bytes, st>>>(p, m.q, m.k, dy);
    return cudaGetLastError();
}
template <int NK>
cudaError_t run_grad(const GradArgs &p, dim3 grid, const DeltaMaps &m, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(delta_grad_kernel<NK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)GradLay<NK>::bytes);
    if (e != cudaSuccess) return e;
    delta_grad_kernel<NK><<<grid, kGradThreads, GradLay<NK>::bytes, st>>>(p, m.q, m.k);
    return cudaGetLastError();
}

int64_t state_bytes(const ssm_delta_args &a) { return (a.dstate <= 64 ? 1 : 2) * (int64_t)kTile; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t delta_tc_bwd_workspace_bytes(const ssm_delta_bwd_args &b) {
    const ssm_delta_args &a = b.fwd;
    const int64_t nsl = (a.headdim + 63) / 64;
    return up256(delta_prep_bytes(a, true)) +
           (size_t)delta_slots(a) * a.nheads * nsl * (2 * state_bytes(a) + 3 * (int64_t)kTile);
}

cudaError_t launch_delta_tc_bwd(const ssm_delta_bwd_args &b, const SeqView &sv, void *ws, cudaStream_t st) {
    const ssm_delta_args &a = b.fwd;
    if ((a.cu_seqlens ? a.nseqs : a.batch) == 0) return cudaSuccess;
    DeltaMaps m;
    CUtensorMap dy;
    const int64_t rows = a.cu_seqlens ? 1 : a.batch, hp = a.nheads * a.headdim;
    if (!delta_maps(a, &m) || !make_map_box(&dy, b.dy, hp, a.seqlen, rows, a.seqlen > 1 ? b.dy_token_stride : hp,
                                            b.dy_batch_stride, false, kQ))
        return cudaErrorInvalidValue;
    uint8_t *prep = static_cast<uint8_t *>(ws);
    Args p;
    p.b = b;
    p.sv = sv;
    p.prep = prep;
    p.nblk = delta_blocks_per_row(a);
    p.slots = delta_slots(a);
    p.R = (int)(a.nheads / a.ngroups);
    p.nsl = (int)((a.headdim + 63) / 64);
    p.units = (p.R * p.nsl + 1) / 2;
    p.rec = Rec{prep + up256(delta_prep_bytes(a, true)), state_bytes(a), p.nsl};
    cudaError_t e = launch_delta_prep(a, sv, m, prep, true, st);
    if (e != cudaSuccess) return e;
    ssm_delta_args f = a;
    f.y = nullptr;
    f.h_final = nullptr;
    e = launch_delta_chain(f, sv, m, prep, &p.rec, st);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.ngroups * p.units), (unsigned)(a.cu_seqlens ? a.nseqs : a.batch));
    const bool dual = p.nsl % 2 != 0;
    timing_begin(st);
    if (a.dstate <= 64) e = dual ? run_chain<64, true>(p, grid, m, dy, st) : run_chain<64, false>(p, grid, m, dy, st);
    else e = dual ? run_chain<128, true>(p, grid, m, dy, st) : run_chain<128, false>(p, grid, m, dy, st);
    timing_end(st);
    if (e != cudaSuccess) return e;
    const GradArgs g{b, sv, p.rec, p.nblk, p.R, p.nsl};
    const dim3 ggrid((unsigned)delta_slots(a), (unsigned)a.ngroups);
    return a.dstate <= 64 ? run_grad<64>(g, ggrid, m, st) : run_grad<128>(g, ggrid, m, st);
}

}  // namespace ssm
