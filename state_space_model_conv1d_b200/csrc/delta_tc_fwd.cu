// delta_tc_fwd.cu -- the gated delta rule in blocks of 64 tokens on the tensor
// cores (bf16 activations, dstate <= 128).
//
// Per block, with the state h entering it and T from delta_prep.cu,
//     R_i = beta_i (v_i - exp(cs_i) h k_i),     U = T R,
//     y_i = scale (exp(cs_i) h q_i + sum_{j<=i} exp(cs_i - cs_j) (q_i . k_j) u_j),
//     h  <- exp(cs_last) h + sum_j exp(cs_last - cs_j) u_j k_j^T.
// A CTA carries 128 state rows (one head of 128, or two 64-row parts of heads
// that share their keys) through its sequence.  Everything is kept transposed,
// state rows in the 128 lanes of tensor memory: R^T, U^T and h are then A
// operands straight from tensor memory, and the chain h -> R -> U -> h never
// touches shared memory.  K serves as a K-major operand (h k) and, the same
// bytes, as an MN-major one (u k^T).
//
// Rounding.  q, k, v are exact bf16.  On the way to the state every factor that
// is not (h, R, T, u) goes as two bf16 parts with fp32 accumulation (relative
// 2^-17 each), so h_final is good to about 1e-5 after any number of blocks.
// What only reaches y (attention weights, u and h of the read-out) is rounded
// to bf16 once, like y itself.
//
// Roles: 8 warps for the chain (two per lane quarter, half of the columns
// each), 4 for the output, one thread each for the chain's MMAs, the output's
// MMAs and the loads (whose warp also computes the gate tables).  A block
// costs three dependent MMA groups; the output's work fills the gaps.
#include <string.h>

#include "delta_tc.cuh"

namespace ssm {

size_t delta_prep_bytes(const ssm_delta_args &a);
cudaError_t launch_delta_prep(const ssm_delta_args &a, const SeqView &sv, void *T, cudaStream_t st);

namespace {

using namespace dtc;

constexpr int kChainWarps = 8, kOutWarps = 4;
constexpr int kThreads = (kChainWarps + kOutWarps + 3) * 32;
// tensor-memory columns
constexpr uint32_t TM_H = 0;       // fp32 state, decayed for the next block
constexpr uint32_t TM_HOP = 128;   // its two bf16 parts (64 columns each)
constexpr uint32_t TM_RU = 256;    // h k, then U
constexpr uint32_t TM_OP = 320;    // R, then the decayed u: two parts of 32 columns
constexpr uint32_t TM_UOP = 384;   // u, high part
constexpr uint32_t TM_O = 416;     // q k, h q, attention x u in turn
constexpr uint32_t kTmemCols = 512;

enum Bar {
    B_FULL0, B_FULL1, B_EMPTY0, B_EMPTY1, B_TAB0, B_TAB1,
    B_H, B_M1, B_R, B_M2, B_U, B_M3,           // the chain
    B_QK, B_PM, B_M4, B_QHREAD, B_M5, B_OREAD, // the output
    B_DRAIN, B_DRAIN2, B_COUNT
};

struct alignas(16) Tab {           // gates of one half of the rows, one block (read as float4)
    float beta[kQ], bg[kQ], w[kQ], gs[kQ], cs[kQ];
    float total;                   // exp(cs_last)
};

struct Aux {
    uint64_t mb[B_COUNT];
    uint32_t tmem;
    int abort;
    Tab tab[2][2];                 // [stage][half]
};

template <int NK, bool DUAL> struct Lay {
    static constexpr uint32_t kKB = NK / 64 * kTile;
    static constexpr uint32_t K = 0, Q = kKB, V = 2 * kKB, T = V + 2 * kTile;
    static constexpr uint32_t stage = T + (DUAL ? 2 : 1) * (uint32_t)kTBytes;
    static constexpr uint32_t PM = 2 * stage, AUX = PM + (DUAL ? 2 : 1) * kTile;
    static constexpr size_t bytes = AUX + sizeof(Aux) + 1024;
    static constexpr uint32_t tx = stage;
};

struct Args {
    ssm_delta_args a;
    SeqView sv;
    const uint8_t *T;
    int64_t nblk;
    int R, nsl, units;             // heads per group, 64-row slices per head, CTAs per group
};

template <int NK, bool DUAL>
__global__ void __launch_bounds__(kThreads, 1)
delta_fwd_kernel(const Args p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v) {
    using L = Lay<NK, DUAL>;
    const ssm_delta_args &a = p.a;
    if (p.sv.err && *p.sv.err != 0) return;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    Aux &ax = *reinterpret_cast<Aux *>(sm + L::AUX);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // the rows: unit -> two halves (head, first row of the head)
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
    if (n == 0) {                              // no token: the state passes through
        if (a.h_final)
            for (int i = 0; i < halves; ++i)
                for (int64_t e = tid; e < min((int64_t)64, P - row0[i]) * N; e += kThreads) {
                    const int64_t at = (((int64_t)s * H + head[i]) * P + row0[i]) * N + e;
                    a.h_final[at] = a.h0 ? a.h0[at] : 0.f;
                }
        return;
    }
    const int64_t slot0 = seq_slot(a.cu_seqlens, s, p.nblk);
    if (warp == 0) tc::tmem_alloc(&ax.tmem, kTmemCols);
    if (tid == 0) {
        constexpr int counts[B_COUNT] = {
            1, 1, 2 + kChainWarps + kOutWarps, 2 + kChainWarps + kOutWarps, 1, 1,
            kChainWarps, 1, kChainWarps, 1, kChainWarps, 1,
            1, kOutWarps, 1, kOutWarps, 1, kOutWarps, 1, 1};
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
    auto wait = [&](int b, uint32_t parity) { return wait_bar(&ax.mb[b], ab, parity, err); };
    const uint32_t sb = tc::smem_u32(sm);

    if (warp < kChainWarps) {
        // ---------------------------------------------------------------- the chain
        const int q = warp & 3, cf = warp >> 2;              // lane quarter, column half
        const int half = q >> 1, r = row0[half] + (q & 1) * 32 + lane;
        const bool live = half < halves && r < P;
        const uint32_t tl = tm + ((uint32_t)(32 * q) << 16);
        const int64_t srow = (((int64_t)s * H + head[half]) * P + r) * N;
        auto arrive_st = [&](int b) {
            tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive(&ax.mb[b]);
        };
        bool ok = wait(B_TAB0, 0);
        // the entering state: NK / 2 columns of this thread's row
#pragma unroll
        for (int b = 0; b < NK / 64; ++b) {
            const int c0 = cf * (NK / 2) + b * 32;
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (live && a.h0 && c0 + i < N) x = *reinterpret_cast<const float4 *>(a.h0 + srow + c0 + i);
                v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
            }
            uint32_t hi_[16], lo_[16];
            split32(v, hi_, lo_);
            tmem_st16(tl + TM_HOP + c0 / 2, hi_);
            tmem_st16(tl + TM_HOP + 64 + c0 / 2, lo_);
            const float d = ax.tab[0][half].total;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= d;
            tmem_st32(tl + TM_H + c0, v);
        }
        arrive_st(B_H);
        for (int c = 0; c < n && ok; ++c) {
            const uint32_t ph = c & 1;
            const int stg = c & 1, nt = (int)min((int64_t)kQ, hi - lo - (int64_t)c * kQ);
            uint8_t *st = sm + stg * L::stage;
            const Tab &tb = ax.tab[stg][half];
            // R = beta (v - exp(cs) h k)
            ok = wait(B_FULL0 + stg, (c >> 1) & 1) && wait(B_TAB0 + stg, (c >> 1) & 1) && wait(B_M1, ph);
            if (!ok) break;
            tc::fence_after_sync();
            float x[32];
            uint32_t hi_[16], lo_[16];
            tc::tmem_ld32(tl + TM_RU + cf * 32, x);
            {
                const __nv_bfloat16 *v =
                    reinterpret_cast<const __nv_bfloat16 *>(st + L::V + half * kTile) + (q & 1) * 32 + lane;
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const int t = cf * 32 + i;
                    const float4 be = *reinterpret_cast<const float4 *>(tb.beta + t);
                    const float4 bg = *reinterpret_cast<const float4 *>(tb.bg + t);
                    const float bb[4] = {be.x, be.y, be.z, be.w}, gg[4] = {bg.x, bg.y, bg.z, bg.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float vv = __bfloat162float(v[(t + e) * 64]);
                        x[i + e] = t + e < nt ? fmaf(-gg[e], x[i + e], bb[e] * vv) : 0.f;
                    }
                }
            }
            if (nt < kQ) {                     // the keys behind the sequence's end may be anything
                for (int i = tid; i < (kQ - nt) * (NK / 8); i += kChainWarps * 32) {
                    const int rr = nt + i / (NK / 8), cc = i % (NK / 8) * 8;
                    *reinterpret_cast<uint4 *>(st + L::K + (cc >> 6) * kTile + swz(rr, cc & 63)) = make_uint4(0, 0, 0, 0);
                }
                tc::fence_proxy_async();
            }
            split32(x, hi_, lo_);
            tmem_st16(tl + TM_OP + cf * 16, hi_);
            tmem_st16(tl + TM_OP + 32 + cf * 16, lo_);
            arrive_st(B_R);
            // u = T R
            ok = wait(B_M2, ph) && (c == 0 || wait(B_M5, ph ^ 1));
            if (!ok) break;
            tc::fence_after_sync();
            tc::tmem_ld32(tl + TM_RU + cf * 32, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) hi_[i] = pack2(x[2 * i], x[2 * i + 1]);
            tmem_st16(tl + TM_UOP + cf * 16, hi_);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 w = *reinterpret_cast<const float4 *>(tb.w + cf * 32 + i);
                x[i] *= w.x; x[i + 1] *= w.y; x[i + 2] *= w.z; x[i + 3] *= w.w;
            }
            split32(x, hi_, lo_);
            tmem_st16(tl + TM_OP + cf * 16, hi_);
            tmem_st16(tl + TM_OP + 32 + cf * 16, lo_);
            arrive_st(B_U);
            if (lane == 0) arrive(&ax.mb[B_EMPTY0 + stg]);
            // h
            const bool last = c + 1 == n;
            ok = wait(B_M3, ph) && wait(B_M4, ph) && (last || wait(B_TAB0 + (stg ^ 1), ((c + 1) >> 1) & 1));
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll
            for (int b = 0; b < NK / 64; ++b) {
                const int c0 = cf * (NK / 2) + b * 32;
                tc::tmem_ld32(tl + TM_H + c0, x);
                if (last) {
                    if (a.h_final && live)
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            if (c0 + i < N)
                                *reinterpret_cast<float4 *>(a.h_final + srow + c0 + i) =
                                    make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                } else {
                    split32(x, hi_, lo_);
                    tmem_st16(tl + TM_HOP + c0 / 2, hi_);
                    tmem_st16(tl + TM_HOP + 64 + c0 / 2, lo_);
                    const float d = ax.tab[stg ^ 1][half].total;
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] *= d;
                    tmem_st32(tl + TM_H + c0, x);
                }
            }
            if (!last) arrive_st(B_H);
        }
    } else if (warp < kChainWarps + kOutWarps) {
        // --------------------------------------------------------------- the output
        const int q = warp - kChainWarps, half = q >> 1, r = row0[half] + (q & 1) * 32 + lane;
        const bool live = half < halves && r < P;
        const uint32_t tl = tm + ((uint32_t)(32 * q) << 16);
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + brow * a.y_batch_stride + lo * a.y_token_stride +
                           (int64_t)head[half] * P + r;
        auto arrive_w = [&](int b) {
            __syncwarp();
            if (lane == 0) arrive(&ax.mb[b]);
        };
        for (int c = 0; c < n; ++c) {
            const uint32_t ph = c & 1;
            const int stg = c & 1, nt = (int)min((int64_t)kQ, hi - lo - (int64_t)c * kQ);
            // attention weights: rows i = 16 q + lane / 4 (+ 8), columns j
            if (!wait(B_TAB0 + stg, (c >> 1) & 1) || !wait(B_QK, ph)) break;
            tc::fence_after_sync();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t qk[16];
                tc::tmem_ld16x256b_x4(tl + TM_O + 32 * b, qk);
                tc::tmem_wait_ld();
#pragma unroll
                for (int hh = 0; hh < (DUAL ? 2 : 1); ++hh) {
                    const float *cs = ax.tab[stg][hh].cs;
                    uint8_t *pm = sm + L::PM + hh * kTile;
#pragma unroll
                    for (int e2 = 0; e2 < 2; ++e2) {
                        const int i = 16 * q + (lane >> 2) + 8 * e2;
                        const float ci = cs[i];
#pragma unroll
                        for (int k8 = 0; k8 < 4; ++k8) {
                            const int j = 32 * b + 8 * k8 + 2 * (lane & 3);
                            const float2 cj = *reinterpret_cast<const float2 *>(cs + j);
                            const float v0 = j <= i && i < nt ? a.scale * ex2(ci - cj.x) * __uint_as_float(qk[4 * k8 + 2 * e2]) : 0.f;
                            const float v1 =
                                j + 1 <= i && i < nt ? a.scale * ex2(ci - cj.y) * __uint_as_float(qk[4 * k8 + 2 * e2 + 1]) : 0.f;
                            *reinterpret_cast<uint32_t *>(pm + swz(i, j)) = pack2(v0, v1);
                        }
                    }
                }
            }
            tc::fence_proxy_async();
            tc::fence_before_sync();
            arrive_w(B_PM);
            // scale exp(cs) h q
            if (!wait(B_M4, ph)) break;
            tc::fence_after_sync();
            float o[64], x[32];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                tc::tmem_ld32(tl + TM_O + 32 * b, x);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 gs = *reinterpret_cast<const float4 *>(ax.tab[stg][half].gs + 32 * b + i);
                    o[32 * b + i] = x[i] * gs.x;
                    o[32 * b + i + 1] = x[i + 1] * gs.y;
                    o[32 * b + i + 2] = x[i + 2] * gs.z;
                    o[32 * b + i + 3] = x[i + 3] * gs.w;
                }
            }
            tc::fence_before_sync();
            arrive_w(B_QHREAD);
            if (lane == 0) arrive(&ax.mb[B_EMPTY0 + stg]);
            if (!wait(B_M5, ph)) break;
            tc::fence_after_sync();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                tc::tmem_ld32(tl + TM_O + 32 * b, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[32 * b + i] += x[i];
            }
            tc::fence_before_sync();
            arrive_w(B_OREAD);
            if (live) {
                __nv_bfloat16 *yc = y + (int64_t)c * kQ * a.y_token_stride;
#pragma unroll
                for (int i = 0; i < kQ; ++i)
                    if (i < nt) yc[i * a.y_token_stride] = __float2bfloat16_rn(o[i]);
            }
        }
    } else if (warp == kChainWarps + kOutWarps) {
        // ----------------------------------------------------- MMAs of the chain
        constexpr uint32_t ID1 = tc::idesc_bf16(128, 64, 0, 0), ID3 = tc::idesc_bf16(128, NK, 0, 1);
        for (int c = 0; c < n; ++c) {
            const uint32_t ph = c & 1;
            const int stg = c & 1;
            const uint32_t st = sb + stg * L::stage;
            const uint64_t dK = tc::desc_sw128(st + L::K, 16, 1024), dKm = tc::desc_sw128(st + L::K, kTile, 1024);
            if (!wait(B_FULL0 + stg, (c >> 1) & 1) || !wait(B_H, ph)) break;
            tc::fence_after_sync();
            if (lane == 0) {
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int kk = 0; kk < NK / 16; ++kk)
                        mma_ts(tm + TM_RU, tm + TM_HOP + part * 64 + kk * 8,
                               dK + (((kk >> 2) * kTile + (kk & 3) * 32) >> 4), ID1, part + kk > 0);
                tc::mma_commit(&ax.mb[B_M1]);
            }
            __syncwarp();
            if (!wait(B_R, ph)) break;
            tc::fence_after_sync();
            if (lane == 0) {
                // U = T R: (R high, T low), (R low, T high), (R high, T high)
#pragma unroll
                for (int hh = 0; hh < (DUAL ? 2 : 1); ++hh) {
                    const uint64_t dT = tc::desc_sw128(st + L::T + hh * (uint32_t)kTBytes, 16, 1024);
#pragma unroll
                    for (int part = 0; part < 3; ++part)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint32_t A = tm + TM_OP + (part == 1 ? 32 : 0) + kk * 8;
                            const uint64_t B = dT + (part == 0 ? kTile >> 4 : 0) + kk * 2;
                            if constexpr (DUAL)
                                mma_ts_lanes(tm + TM_RU, A, B, ID1, part + kk > 0, hh ? ~0u : 0u, hh ? 0u : ~0u);
                            else
                                mma_ts(tm + TM_RU, A, B, ID1, part + kk > 0);
                        }
                }
                tc::mma_commit(&ax.mb[B_M2]);
            }
            __syncwarp();
            if (!wait(B_U, ph)) break;
            tc::fence_after_sync();
            if (lane == 0) {
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ts(tm + TM_H, tm + TM_OP + part * 32 + kk * 8, dKm + kk * 128, ID3, 1);
                tc::mma_commit(&ax.mb[B_M3]);
                tc::mma_commit(&ax.mb[B_EMPTY0 + stg]);
            }
            __syncwarp();
        }
    } else if (warp == kChainWarps + kOutWarps + 1) {
        // ---------------------------------------------------- MMAs of the output
        constexpr uint32_t ID1 = tc::idesc_bf16(128, 64, 0, 0), IDQ = tc::idesc_bf16(64, 64, 0, 0);
        auto qk = [&](int c) {
            const uint32_t st = sb + (c & 1) * L::stage;
            const uint64_t dQ = tc::desc_sw128(st + L::Q, 16, 1024), dK = tc::desc_sw128(st + L::K, 16, 1024);
            if (!wait(B_FULL0 + (c & 1), (c >> 1) & 1)) return false;
            tc::fence_after_sync();
            if (lane == 0) {
#pragma unroll
                for (int kk = 0; kk < NK / 16; ++kk) {
                    const uint32_t o = ((kk >> 2) * kTile + (kk & 3) * 32) >> 4;
                    tc::mma_bf16(tm + TM_O, dQ + o, dK + o, IDQ, kk > 0);
                }
                tc::mma_commit(&ax.mb[B_QK]);
            }
            __syncwarp();
            return true;
        };
        bool ok = qk(0);
        for (int c = 0; c < n && ok; ++c) {
            const uint32_t ph = c & 1;
            const int stg = c & 1;
            const uint64_t dQ = tc::desc_sw128(sb + stg * L::stage + L::Q, 16, 1024);
            ok = wait(B_H, ph) && wait(B_PM, ph);
            if (!ok) break;
            tc::fence_after_sync();
            if (lane == 0) {
#pragma unroll
                for (int kk = 0; kk < NK / 16; ++kk)
                    mma_ts(tm + TM_O, tm + TM_HOP + kk * 8, dQ + (((kk >> 2) * kTile + (kk & 3) * 32) >> 4), ID1, kk > 0);
                tc::mma_commit(&ax.mb[B_M4]);
                tc::mma_commit(&ax.mb[B_EMPTY0 + stg]);
            }
            __syncwarp();
            ok = wait(B_QHREAD, ph) && wait(B_U, ph);
            if (!ok) break;
            tc::fence_after_sync();
            if (lane == 0) {
#pragma unroll
                for (int hh = 0; hh < (DUAL ? 2 : 1); ++hh) {
                    const uint64_t dP = tc::desc_sw128(sb + L::PM + hh * kTile, 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if constexpr (DUAL)
                            mma_ts_lanes(tm + TM_O, tm + TM_UOP + kk * 8, dP + kk * 2, ID1, kk > 0, hh ? ~0u : 0u,
                                         hh ? 0u : ~0u);
                        else
                            mma_ts(tm + TM_O, tm + TM_UOP + kk * 8, dP + kk * 2, ID1, kk > 0);
                }
                tc::mma_commit(&ax.mb[B_M5]);
            }
            __syncwarp();
            ok = wait(B_OREAD, ph);
            if (ok && c + 1 < n) {
                tc::fence_after_sync();
                ok = qk(c + 1);
            }
        }
    } else {
        // --------------------------------------------------- loads and gate tables
        int issued = 0;
        for (int c = 0; c < n; ++c) {
            const int stg = c & 1;
            const int64_t t0 = lo + (int64_t)c * kQ;
            const int nt = (int)min((int64_t)kQ, hi - t0);
            float gv[2][2], bv[2][2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = lane + 32 * e;
                    const bool in = t < nt && (hh == 0 || head[1] != head[0]);
                    gv[hh][e] = in ? a.g[brow * a.g_batch_stride + (t0 + t) * a.g_token_stride + head[hh]] : 0.f;
                    bv[hh][e] = in ? a.beta[brow * a.beta_batch_stride + (t0 + t) * a.beta_token_stride + head[hh]] : 0.f;
                }
            if (c >= 2 && !wait(B_EMPTY0 + stg, ((c >> 1) - 1) & 1)) break;
            uint8_t *st = sm + stg * L::stage;
            if (lane == 0) {
                uint64_t *mb = &ax.mb[B_FULL0 + stg];
                tc::mbar_expect_tx(mb, L::tx);
#pragma unroll
                for (int x = 0; x < NK / 64; ++x) {
                    tma_load_4d(st + L::K + x * kTile, &tm_k, 64 * x, grp, (int)t0, (int)brow, mb);
                    tma_load_4d(st + L::Q + x * kTile, &tm_q, 64 * x, grp, (int)t0, (int)brow, mb);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    tc::tma_load_3d(st + L::V + i * kTile, &tm_v, (int)(head[i] * P + row0[i]), (int)t0, (int)brow, mb);
#pragma unroll
                for (int i = 0; i < (DUAL ? 2 : 1); ++i)
                    bulk_load(st + L::T + i * (uint32_t)kTBytes, p.T + ((slot0 + c) * H + head[i]) * kTBytes,
                              (uint32_t)kTBytes, mb);
            }
            issued = c + 1;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                Tab &tb = ax.tab[stg][hh];
                if (hh == 1 && head[1] == head[0]) {
                    gv[1][0] = gv[0][0]; gv[1][1] = gv[0][1];
                    bv[1][0] = bv[0][0]; bv[1][1] = bv[0][1];
                }
                double cs[2], last;
                block_cs(fmaxf(gv[hh][0], kMinLogDecay), fmaxf(gv[hh][1], kMinLogDecay), cs[0], cs[1], last);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = lane + 32 * e;
                    const float ec = exp_d(cs[e]);
                    tb.beta[t] = bv[hh][e];
                    tb.bg[t] = bv[hh][e] * ec;
                    tb.w[t] = exp_d(last - cs[e]);
                    tb.gs[t] = a.scale * ec;
                    tb.cs[t] = (float)(cs[e] * 1.4426950408889634);
                }
                if (lane == 0) tb.total = exp_d(last);
            }
            __syncwarp();
            if (lane == 0) arrive(&ax.mb[B_TAB0 + stg]);
        }
        if (*ab && lane == 0)                  // copies in flight land before the CTA ends
            for (int c = max(0, issued - 2); c < issued; ++c) tc::mbar_wait(&ax.mb[B_FULL0 + (c & 1)], (c >> 1) & 1, 1u << 22);
    }
    if (*ab && lane == 0 && (warp == kChainWarps + kOutWarps || warp == kChainWarps + kOutWarps + 1)) {
        // after a wait that ran out: the MMAs this thread issued complete before tensor memory is freed
        uint64_t *mb = &ax.mb[warp == kChainWarps + kOutWarps ? B_DRAIN : B_DRAIN2];
        tc::mma_commit(mb);
        tc::mbar_wait(mb, 0, 1u << 22);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tm, kTmemCols);
    }
}

template <int NK, bool DUAL>
cudaError_t run(const Args &p, dim3 grid, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(delta_fwd_kernel<NK, DUAL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Lay<NK, DUAL>::bytes);
    if (e != cudaSuccess) return e;
    delta_fwd_kernel<NK, DUAL><<<grid, kThreads, Lay<NK, DUAL>::bytes, st>>>(p, q, k, v);
    return cudaGetLastError();
}

}  // namespace

bool delta_tc_shape(const ssm_delta_args &a) {
    return a.dtype == SSM_BF16 && a.dstate <= 128 && a.dstate % 8 == 0 && a.headdim % 8 == 0;
}
bool delta_tc_ok(const ssm_delta_args &a) {
    auto al = [](const void *p, int64_t bs, int64_t ts) {
        return ((uintptr_t)p % 16) == 0 && bs % 8 == 0 && ts % 8 == 0;
    };
    return delta_tc_shape(a) && a.seqlen > 0 && al(a.q, a.q_batch_stride, a.q_token_stride) &&
           al(a.k, a.k_batch_stride, a.k_token_stride) && al(a.v, a.v_batch_stride, a.v_token_stride) &&
           al(a.h0, 0, 0) && al(a.h_final, 0, 0);
}
size_t delta_tc_workspace_bytes(const ssm_delta_args &a) { return delta_prep_bytes(a); }

cudaError_t launch_delta_tc(const ssm_delta_args &a, const SeqView &sv, void *ws, cudaStream_t st) {
    const int64_t nseq = a.cu_seqlens ? a.nseqs : a.batch;
    if (nseq == 0) return cudaSuccess;
    Args p;
    p.a = a;
    p.sv = sv;
    p.T = static_cast<const uint8_t *>(ws);
    p.nblk = delta_blocks_per_row(a);
    p.R = (int)(a.nheads / a.ngroups);
    p.nsl = (int)((a.headdim + 63) / 64);
    p.units = (p.R * p.nsl + 1) / 2;
    const int64_t rows = a.cu_seqlens ? 1 : a.batch;
    CUtensorMap q, k, v;
    if (!make_map_group(&q, a.q, a.dstate, a.ngroups, a.seqlen, rows, a.q_token_stride, a.q_batch_stride) ||
        !make_map_group(&k, a.k, a.dstate, a.ngroups, a.seqlen, rows, a.k_token_stride, a.k_batch_stride) ||
        !make_map_box(&v, a.v, a.nheads * a.headdim, a.seqlen, rows,
                      a.seqlen > 1 ? a.v_token_stride : a.nheads * a.headdim, a.v_batch_stride, false, kQ))
        return cudaErrorInvalidValue;
    cudaError_t e = launch_delta_prep(a, sv, ws, st);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.ngroups * p.units), (unsigned)nseq);
    const bool dual = p.nsl % 2 != 0;
    timing_begin(st);
    if (a.dstate <= 64) e = dual ? run<64, true>(p, grid, q, k, v, st) : run<64, false>(p, grid, q, k, v, st);
    else e = dual ? run<128, true>(p, grid, q, k, v, st) : run<128, false>(p, grid, q, k, v, st);
    timing_end(st);
    return e;
}

}  // namespace ssm
