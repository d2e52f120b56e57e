// delta_tc_fwd.cu -- the gated delta rule in blocks of 64 tokens on the tensor
// cores (bf16 activations, dstate <= 128).
//
// Per block, with the state h entering it and T and the attention weights from
// delta_prep.cu,
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
// 2^-17 each): h_final is off by 3.5e-6 of its norm after nine blocks, 1.2e-5
// with keys alike and beta 2.  Of what only reaches y the attention weights are
// rounded to bf16 once, like y itself: y is off by 2.1e-3 to 2.3e-3 of its norm,
// and rounding the exact y gives 1.7e-3.  Their low part would make y's products
// half as many again and its operand 16 KB instead of 8 a block and head, written
// by a pre-pass that is bound by shared memory, for a y that is bf16 itself.  u
// goes as two parts there too (with its high part alone y was off by 2.6e-3, in
// 1.5 % less time).
//
// Roles: 8 warps for the chain (two per lane quarter, half of the columns
// each), 4 for the output (one thread of them issues its product), one thread
// for the chain's MMAs and one warp for the loads and the gate tables.  A block costs three
// dependent groups of MMAs (h k with h q beside it, T R, the state's update)
// with a pass over registers between them; each pass hands over its first half
// as soon as it is written, so that the MMAs of that half overlap the second.
// An MMA of 128 rows takes about 65 cycles whether it has 64 columns or
// 128, so products that share the A operand are joined: K and Q lie one behind
// the other and make one operand of 128 rows, and so do the two T of a CTA
// whose halves are different heads.
//
// 4 x 4096 tokens, 32 heads of P 128, N 128: 232 us, 64 blocks one after the
// other in 128 CTAs, 3.6 us (6.6k cycles) a block: the chain's latency, 36 MMAs
// of about 100 cycles and the passes between them.  28301 packed tokens, 64 heads
// of P 64, two of them in a CTA: 443 us, 7.2k cycles a block.  (With the output's
// product in the MMA warp, whose waits then queue up behind the products already
// issued, it was 17 and 22 us more; with waits whose outcome each lane keeps for
// itself 8 and 7 us more.)  The token-by-token form takes 15 times as long
// on the first call.
#include <string.h>

#include "delta_tc.cuh"
#include "delta_tc.h"

namespace ssm {

namespace {

using namespace dtc;

// A warp reaches the tensor-memory lanes of its number modulo 4.
constexpr int kChainWarps = 8, kOutWarps = 4;
constexpr int kOut0 = kChainWarps, kMmaWarp = kOut0 + kOutWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = (kLoadWarp + 1) * 32;
static_assert(kOut0 % 4 == 0, "lane quarters");
// tensor-memory columns
constexpr uint32_t TM_H = 0;       // fp32 state, decayed for the next block
constexpr uint32_t TM_HOP = 128;   // its two bf16 parts: per half of the pass 32 high, 32 low columns
constexpr uint32_t TM_RU = 256;    // h k, then U (two heads: in 128 columns), then u (per half 16 columns high, 16 low)
constexpr uint32_t TM_HQ = 320;    // h q
constexpr uint32_t TM_O = 384;     // scale exp(cs) h q, to which attention x u is added
constexpr uint32_t TM_OP = 448;    // R, then the decayed u: two parts of 32 columns
constexpr uint32_t kTmemCols = 512;

enum Bar {
    B_FULL0, B_FULL1, B_EMPTY0, B_EMPTY1, B_TAB0, B_TAB1,
    B_H0, B_H1, B_M1, B_R0, B_R1, B_M2, B_U0, B_U1, B_UOP, B_M3,    // the chain (halves 0 and 1 of a pass)
    B_HQ, B_M5,                                                     // the output
    B_DRAIN, B_DRAIN2, B_COUNT
};

// Operand columns of the state's part (0 high, 1 low): states 32 b .. 32 b + 31 of column half cf.
SSM_DEVINL uint32_t hop(int cf, int b, int part) { return TM_HOP + 64 * b + 32 * part + 16 * cf; }

struct alignas(16) Tab {           // gates of one half of the rows, one block (read as float4)
    float beta[kQ], bg[kQ], w[kQ], gs[kQ];
    float total;                   // exp(cs_last)
};

struct Aux {
    uint64_t mb[B_COUNT];
    uint32_t tmem;
    int abort;
    Tab tab[2][2];                 // [stage][half]
};

template <int NK, bool DUAL> struct Lay {
    static constexpr uint32_t kKB = NK / 64 * 2 * kTile;             // per K-atom: 64 rows of K, 64 rows of Q
    static constexpr uint32_t K = 0, V = kKB, T = V + 2 * kTile;      // T: high parts of both heads, low parts
    static constexpr uint32_t kTPart = (DUAL ? 2 : 1) * kTile;
    static constexpr uint32_t PM = T + 2 * kTPart, stage = PM + kTPart;
    static constexpr uint32_t Y = 2 * stage, AUX = Y + 2 * kTile;
    static constexpr size_t bytes = AUX + sizeof(Aux) + 1024;
    static constexpr uint32_t tx(bool st) { return st ? PM : stage; }
};

struct Args {
    ssm_delta_args a;
    SeqView sv;
    const uint8_t *prep;           // delta_prep.cu: [slot][H][kHeadBytes]
    int64_t nblk, slots;
    int R, nsl, units;             // heads per group, 64-row slices per head, CTAs per group
    Rec rec;                       // the states' pass of the backward: where u and the states go
};

// ST: the states' pass of the backward: no output, but every block's entering
// state and u are kept (attention weights are neither loaded nor used).
template <int NK, bool DUAL, bool ST>
__global__ void __launch_bounds__(kThreads, 1)
delta_fwd_kernel(const Args p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v) {
    using L = Lay<NK, DUAL>;
    const ssm_delta_args &a = p.a;
    if (p.sv.err && *p.sv.err != 0) return;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = smem_1024(raw);
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
    if (!SSM_BOUNDS(slot0 + n - 1, p.slots, BS_DELTA_SLOT) || !SSM_BOUNDS(max(head[0], head[1]), H, BS_DELTA_HEAD) ||
        !SSM_BOUNDS(max(row0[0], row0[1]), P, BS_DELTA_STATE)) return;
    if (warp == 0) tc::tmem_alloc(&ax.tmem, kTmemCols);
    if (tid == 0) {
        constexpr int kEmpty = 1 + kChainWarps + (ST ? 0 : 1 + kOutWarps);
        constexpr int counts[B_COUNT] = {
            1, 1, kEmpty, kEmpty, 1, 1,
            kChainWarps, kChainWarps, 1, kChainWarps, kChainWarps, 1, kChainWarps, kChainWarps, kChainWarps, 1,
            kOutWarps, 1,
            1, 1};
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
    int issued = 0;                            // blocks whose loads the load warp has issued

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
        // the states' pass: values of this thread's row in a tile of block c, 16 bytes at a time
        const int rr = (q & 1) * 32 + lane;
        auto keep = [&](int c, int64_t off, int col, const float *v, int n8) {
            if (half >= halves) return;
            uint8_t *rec = p.rec.at(slot0 + c, H, head[half], row0[half] / 64);
            for (int k = 0; k < n8; ++k) {
                uint4 o = make_uint4(0, 0, 0, 0);
                const float *f = v + 8 * k;
                if (live) o = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
                *reinterpret_cast<uint4 *>(rec + off + rec_off(rr, col + 8 * k)) = o;
            }
        };
        bool ok = wait(B_TAB0, 0);
        // the entering state: NK / 2 columns of this thread's row
#pragma unroll 1
        for (int e = 0; e < NK / 32; ++e) {
            const int c0 = cf * (NK / 2) + e * 16;
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (live && a.h0 && c0 + i < N) x = *reinterpret_cast<const float4 *>(a.h0 + srow + c0 + i);
                v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
            }
            st_split16(tl + hop(cf, e >> 1, 0) + 8 * (e & 1), tl + hop(cf, e >> 1, 1) + 8 * (e & 1), v);
            if (ST) keep(0, 0, c0, v, 2);
            const float d = ax.tab[0][half].total;
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= d;
            tmem_st16f(tl + TM_H + c0, v);
        }
        arrive_st(B_H0);
        if (lane == 0) arrive(&ax.mb[B_H1]);
        for (int c = 0; c < n && ok; ++c) {
            const uint32_t ph = c & 1;
            const int stg = c & 1, nt = (int)min((int64_t)kQ, hi - lo - (int64_t)c * kQ);
            uint8_t *st = sm + stg * L::stage;
            const Tab &tb = ax.tab[stg][half];
            // R = beta (v - exp(cs) h k); what does not need h while the product runs
            ok = wait(B_FULL0 + stg, (c >> 1) & 1) && wait(B_TAB0 + stg, (c >> 1) & 1);
            if (!ok) break;
            const int t0 = cf * 32;
            float x[32];
            uint32_t raw_[32];
            {
                float bv[32], bg[32];
                const __nv_bfloat16 *v =
                    reinterpret_cast<const __nv_bfloat16 *>(st + L::V + half * kTile) + t0 * 64 + (q & 1) * 32 + lane;
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 be = *reinterpret_cast<const float4 *>(tb.beta + t0 + i);
                    const float4 g4 = *reinterpret_cast<const float4 *>(tb.bg + t0 + i);
                    bv[i] = be.x * __bfloat162float(v[i * 64]);
                    bv[i + 1] = be.y * __bfloat162float(v[(i + 1) * 64]);
                    bv[i + 2] = be.z * __bfloat162float(v[(i + 2) * 64]);
                    bv[i + 3] = be.w * __bfloat162float(v[(i + 3) * 64]);
                    bg[i] = g4.x; bg[i + 1] = g4.y; bg[i + 2] = g4.z; bg[i + 3] = g4.w;
                }
                ok = wait(B_M1, ph);
                if (!ok) break;
                tc::fence_after_sync();
                // all of h k is read before the first half of R lets U overwrite it
                tmem_ld32_start(tl + TM_RU + t0, raw_);
                if (nt < kQ) {                 // the keys behind the sequence's end may be anything
                    for (int i = tid; i < (kQ - nt) * (NK / 8); i += kChainWarps * 32) {
                        const int rr = nt + i / (NK / 8), cc = i % (NK / 8) * 8;
                        *reinterpret_cast<uint4 *>(st + L::K + (cc >> 6) * 2 * kTile + swz(rr, cc & 63)) =
                            make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_proxy_async();
                }
                tmem_ld32_wait(raw_, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = fmaf(-bg[i], x[i], bv[i]);
            }
            if (nt < kQ)                       // v and h k of the rows behind the end may be anything
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (t0 + i >= nt) x[i] = 0.f;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                st_split16(tl + TM_OP + t0 / 2 + 8 * b, tl + TM_OP + 32 + t0 / 2 + 8 * b, x + 16 * b);
                arrive_st(B_R0 + b);
            }
            // u = T R
            {
                float w[32];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 w4 = *reinterpret_cast<const float4 *>(tb.w + t0 + i);
                    w[i] = w4.x; w[i + 1] = w4.y; w[i + 2] = w4.z; w[i + 3] = w4.w;
                }
                ok = wait(B_M2, ph);
                if (!ok) break;
                tc::fence_after_sync();
                tmem_ld32_start(tl + TM_RU + (DUAL && half ? 64 : 0) + t0, raw_);
                tmem_ld32_wait(raw_, x);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float y[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] = w[16 * b + i] * x[16 * b + i];
                    st_split16(tl + TM_OP + t0 / 2 + 8 * b, tl + TM_OP + 32 + t0 / 2 + 8 * b, y);
                    arrive_st(B_U0 + b);
                }
            }
            // u for the output in two parts, over the 32 columns of U that this warp has read
            if constexpr (ST) {
                keep(c, p.rec.u(), t0, x, 4);
            } else {
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    st_split16(tl + TM_RU + t0 + 8 * b, tl + TM_RU + t0 + 16 + 8 * b, x + 16 * b);
                arrive_st(B_UOP);
            }
            if (lane == 0) arrive(&ax.mb[B_EMPTY0 + stg]);
            // h
            const bool last = c + 1 == n;
            ok = last || wait(B_TAB0 + (stg ^ 1), ((c + 1) >> 1) & 1);
            if (!ok) break;
            const float d = last ? 1.f : ax.tab[stg ^ 1][half].total;
            ok = wait(B_M3, ph);
            if (!ok) break;
            tc::fence_after_sync();
            float h1[32];
            uint32_t raw1[32];
            tmem_ld32_start(tl + TM_H + cf * (NK / 2), raw_);
            if (NK == 128) tmem_ld32_start(tl + TM_H + cf * (NK / 2) + 32, raw1);
            tmem_ld32_wait(raw_, x);
            if (NK == 128) tmem_ld32_wait(raw1, h1);
            if (last) {
                if (a.h_final && live)
#pragma unroll
                    for (int b = 0; b < NK / 64; ++b)
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const int c0 = cf * (NK / 2) + b * 32 + i;
                            const float *f = (b ? h1 : x) + i;
                            if (c0 < N)
                                *reinterpret_cast<float4 *>(a.h_final + srow + c0) = make_float4(f[0], f[1], f[2], f[3]);
                        }
                break;
            }
#pragma unroll
            for (int b = 0; b < NK / 64; ++b) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    st_split16(tl + hop(cf, b, 0) + 8 * e, tl + hop(cf, b, 1) + 8 * e, (b ? h1 : x) + 16 * e);
                arrive_st(B_H0 + b);
            }
            if (NK == 64 && lane == 0) arrive(&ax.mb[B_H1]);
            if (ST) {
                keep(c + 1, 0, cf * (NK / 2), x, 4);
                if (NK == 128) keep(c + 1, 0, cf * (NK / 2) + 32, h1, 4);
            }
            // decayed for the next block's update; R, handed over later, covers these stores
#pragma unroll
            for (int b = 0; b < NK / 64; ++b) {
                float *f = b ? h1 : x;
#pragma unroll
                for (int i = 0; i < 32; ++i) f[i] *= d;
                tmem_st32(tl + TM_H + cf * (NK / 2) + b * 32, b ? h1 : x);
            }
        }
    } else if (warp < kMmaWarp) {
        // --------------------------------------------------------------- the output
        const int q = warp - kOut0, half = q >> 1;
        const uint32_t tl = tm + ((uint32_t)(32 * q) << 16);
        const int ch = (32 * q + lane) & 15, yh = ch >> 3;
        const bool in = yh < halves && row0[yh] + (ch & 7) * 8 < P;
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + brow * a.y_batch_stride + lo * a.y_token_stride +
                           (int64_t)head[yh] * P + row0[yh] + (ch & 7) * 8;
        __nv_bfloat16 *ys = reinterpret_cast<__nv_bfloat16 *>(sm + L::Y);
        for (int c = 0; !ST && c < n; ++c) {
            const uint32_t ph = c & 1;
            const int stg = c & 1, nt = (int)min((int64_t)kQ, hi - lo - (int64_t)c * kQ);
            float x[32];
            // scale exp(cs) h q into the accumulator of attention x u
            bool ok = wait(B_TAB0 + stg, (c >> 1) & 1) && wait(B_M1, ph);
            tc::fence_after_sync();
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                tc::tmem_ld32(tl + TM_HQ + 32 * b, x);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 gs = *reinterpret_cast<const float4 *>(ax.tab[stg][half].gs + 32 * b + i);
                    x[i] *= gs.x; x[i + 1] *= gs.y; x[i + 2] *= gs.z; x[i + 3] *= gs.w;
                }
                tmem_st32(tl + TM_O + 32 * b, x);
            }
            tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                arrive(&ax.mb[B_HQ]);
                arrive(&ax.mb[B_EMPTY0 + stg]);
            }
            // attention x u, issued here: in the MMA warp its waits would queue up behind the chain's products
            if (q == 0) {
                ok = ok && wait(B_FULL0 + stg, (c >> 1) & 1) && wait(B_HQ, ph) && wait(B_UOP, ph);
                if (ok && lane == 0) {
                    tc::fence_after_sync();
                    constexpr uint32_t ID5 = tc::idesc_bf16(128, 64, 0, 0);
                    const uint64_t dP = tc::desc_sw128(sb + stg * L::stage + L::PM, 16, 1024);
#pragma unroll
                    for (int hh = 0; hh < (DUAL ? 2 : 1); ++hh)
#pragma unroll
                        for (int kp = 0; kp < 8; ++kp) {
                            const int kk = kp & 3;
                            const uint32_t A = tm + TM_RU + (kk >> 1) * 32 + (kk & 1) * 8 + (kp >> 2) * 16;
                            const uint64_t B = dP + hh * (kTile >> 4) + kk * 2;
                            if constexpr (DUAL)
                                mma_ts_lanes(tm + TM_O, A, B, ID5, 1, hh ? ~0u : 0u, hh ? 0u : ~0u);
                            else
                                mma_ts(tm + TM_O, A, B, ID5, 1);
                        }
                    tc::mma_commit(&ax.mb[B_M5]);
                    tc::mma_commit(&ax.mb[B_EMPTY0 + stg]);
                }
                __syncwarp();
            }
            ok = ok && wait(B_M5, ph);
            tc::fence_after_sync();
            // y by way of shared memory: whole 16-byte pieces of token rows
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                tc::tmem_ld32(tl + TM_O + 32 * b, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) ys[(32 * b + i) * 128 + 32 * q + lane] = __float2bfloat16_rn(x[i]);
            }
            if (!bar_all<128>(ok)) break;
            if (in) {
                __nv_bfloat16 *yc = y + (int64_t)c * kQ * a.y_token_stride;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = 2 * q + (lane >> 4) + 8 * i;
                    if (t < nt && SSM_BOUNDS(lo + (int64_t)c * kQ + t, a.seqlen, BS_DELTA_OUT))
                        *reinterpret_cast<uint4 *>(yc + t * a.y_token_stride) =
                            *reinterpret_cast<const uint4 *>(ys + t * 128 + ch * 8);
                }
            }
            asm volatile("bar.sync 1, 128;\n" ::: "memory");
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------------ MMAs
        constexpr uint32_t ID1 = tc::idesc_bf16(128, 128, 0, 0), ID2 = tc::idesc_bf16(128, DUAL ? 128 : 64, 0, 0),
                           ID3 = tc::idesc_bf16(128, NK, 0, 1);
        bool ok = true;
        for (int c = 0; c < n && ok; ++c) {
            const uint32_t ph = c & 1;
            const int stg = c & 1;
            const uint32_t st = sb + stg * L::stage;
            const uint64_t dK = tc::desc_sw128(st + L::K, 16, 1024), dKm = tc::desc_sw128(st + L::K, 2 * kTile, 1024);
            const uint64_t dT = tc::desc_sw128(st + L::T, 16, 1024);
            // h k and h q, once the last block's attention product has used u (it follows the reading of h q)
            ok = wait(B_FULL0 + stg, (c >> 1) & 1) && (ST || c == 0 || wait(B_M5, ph ^ 1));
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                ok = ok && wait(B_H0 + b, ph);
                if (!ok) break;
                tc::fence_after_sync();
                if (lane == 0) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k4 = 0; k4 < NK / 32; ++k4) {
                            // the first half of a pass: states 32 cf ... of each column half
                            const int kk = NK == 64 ? 2 * b + k4 : (k4 >> 1) * 4 + 2 * b + (k4 & 1);
                            mma_ts(tm + TM_RU, tm + hop(NK == 64 ? b : k4 >> 1, NK == 64 ? 0 : b, part) + (k4 & 1) * 8,
                                   dK + (((kk >> 2) * 2 * kTile + (kk & 3) * 32) >> 4), ID1, b + part + k4 > 0);
                        }
                    if (b) tc::mma_commit(&ax.mb[B_M1]);
                }
                __syncwarp();
            }
            // U = T R: (R high, T low), (R low, T high), (R high, T high)
            ok = ok && (!DUAL || ST || wait(B_HQ, ph));
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                ok = ok && wait(B_R0 + b, ph);
                if (!ok) break;
                tc::fence_after_sync();
                if (lane == 0) {
#pragma unroll
                    for (int part = 0; part < 3; ++part)
#pragma unroll
                        for (int k2 = 0, kk = b; k2 < 2; ++k2, kk += 2)
                            mma_ts(tm + TM_RU, tm + TM_OP + (part == 1 ? 32 : 0) + kk * 8,
                                   dT + (part == 0 ? L::kTPart >> 4 : 0) + kk * 2, ID2, b + part + kk > 0);
                    if (b) tc::mma_commit(&ax.mb[B_M2]);
                }
                __syncwarp();
            }
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                ok = ok && wait(B_U0 + b, ph);
                if (!ok) break;
                tc::fence_after_sync();
                if (lane == 0) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k2 = 0, kk = b; k2 < 2; ++k2, kk += 2)
                            mma_ts(tm + TM_H, tm + TM_OP + part * 32 + kk * 8, dKm + kk * 128, ID3, 1);
                    if (b) {
                        tc::mma_commit(&ax.mb[B_M3]);
                        tc::mma_commit(&ax.mb[B_EMPTY0 + stg]);
                    }
                }
                __syncwarp();
            }
        }
    } else {
        // --------------------------------------------------- loads and gate tables
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
                    if (ST) bv[hh][e] = bwd_beta(bv[hh][e]);
                }
            if (c >= 2 && !wait(B_EMPTY0 + stg, ((c >> 1) - 1) & 1)) break;
            uint8_t *st = sm + stg * L::stage;
            if (lane == 0) {
                uint64_t *mb = &ax.mb[B_FULL0 + stg];
                tc::mbar_expect_tx(mb, L::tx(ST));
#pragma unroll
                for (int x = 0; x < NK / 64; ++x) {
                    tma_load_4d(st + L::K + x * 2 * kTile, &tm_k, 64 * x, grp, (int)t0, (int)brow, mb);
                    tma_load_4d(st + L::K + x * 2 * kTile + kTile, &tm_q, 64 * x, grp, (int)t0, (int)brow, mb);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    tc::tma_load_3d(st + L::V + i * kTile, &tm_v, (int)(head[i] * P + row0[i]), (int)t0, (int)brow, mb);
#pragma unroll
                for (int i = 0; i < (DUAL ? 2 : 1); ++i)
#pragma unroll
                    for (int part = 0; part < (ST ? 2 : 3); ++part)       // T high, T low, attention weights
                        bulk_load(st + L::T + part * L::kTPart + i * kTile,
                                  p.prep + ((slot0 + c) * H + head[i]) * (ST ? kHeadBytesBwd : kHeadBytes) + part * kTile,
                                  kTile, mb);
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
    if (*ab) {
        // A wait ran out, here or in a warp that came later than this one: what is in flight (copies, MMAs, stores to
        // tensor memory) lands before tensor memory is freed and the CTA ends.
        if (warp < kMmaWarp) tmem_wait_st();
        if (warp == kLoadWarp && lane == 0)
            for (int c = max(0, issued - 2); c < issued; ++c) tc::mbar_wait(&ax.mb[B_FULL0 + (c & 1)], (c >> 1) & 1, 1u << 22);
        if (lane == 0 && (warp == kMmaWarp || warp == kOut0)) {
            const int b = warp == kMmaWarp ? B_DRAIN : B_DRAIN2;
            tc::mma_commit(&ax.mb[b]);
            tc::mbar_wait(&ax.mb[b], 0, 1u << 22);
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

template <int NK, bool DUAL, bool ST>
cudaError_t run(const Args &p, dim3 grid, const DeltaMaps &m, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(delta_fwd_kernel<NK, DUAL, ST>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Lay<NK, DUAL>::bytes);
    if (e != cudaSuccess) return e;
    delta_fwd_kernel<NK, DUAL, ST><<<grid, kThreads, Lay<NK, DUAL>::bytes, st>>>(p, m.q, m.k, m.v);
    return cudaGetLastError();
}

}  // namespace

bool delta_tc_shape(const ssm_delta_args &a) {
    return a.dtype == SSM_BF16 && a.dstate <= 128 && a.dstate % 8 == 0 && a.headdim % 8 == 0 && a.nheads <= 65535 &&
           a.nheads * a.headdim <= INT32_MAX;
}
namespace {
bool al16(const void *p, int64_t bs = 0, int64_t ts = 0) { return ((uintptr_t)p % 16) == 0 && bs % 8 == 0 && ts % 8 == 0; }
}  // namespace
bool delta_tc_ok(const ssm_delta_args &a) {
    return delta_tc_shape(a) && a.seqlen > 0 && al16(a.q, a.q_batch_stride, a.q_token_stride) &&
           al16(a.k, a.k_batch_stride, a.k_token_stride) && al16(a.v, a.v_batch_stride, a.v_token_stride) &&
           al16(a.y, a.y_batch_stride, a.y_token_stride) && al16(a.h0) && al16(a.h_final);
}
bool delta_tc_bwd_ok(const ssm_delta_bwd_args &b) {
    ssm_delta_args f = b.fwd;
    f.y = const_cast<void *>(b.dy);
    f.y_batch_stride = b.dy_batch_stride;
    f.y_token_stride = b.dy_token_stride;
    f.h_final = nullptr;
    return delta_tc_ok(f) && al16(b.dh_final) && al16(b.dq) && al16(b.dk) && al16(b.dv) && al16(b.dh0);
}
size_t delta_tc_workspace_bytes(const ssm_delta_args &a) { return delta_prep_bytes(a, false); }

bool delta_maps(const ssm_delta_args &a, DeltaMaps *m) {
    const int64_t rows = a.cu_seqlens ? 1 : a.batch, hp = a.nheads * a.headdim;
    return make_map_group(&m->q, a.q, a.dstate, a.ngroups, a.seqlen, rows, a.q_token_stride, a.q_batch_stride) &&
           make_map_group(&m->k, a.k, a.dstate, a.ngroups, a.seqlen, rows, a.k_token_stride, a.k_batch_stride) &&
           make_map_box(&m->v, a.v, hp, a.seqlen, rows, a.seqlen > 1 ? a.v_token_stride : hp, a.v_batch_stride, false,
                        dtc::kQ);
}

cudaError_t launch_delta_chain(const ssm_delta_args &a, const SeqView &sv, const DeltaMaps &m, const void *prep,
                               const dtc::Rec *rec, cudaStream_t st) {
    Args p;
    p.a = a;
    p.sv = sv;
    p.prep = static_cast<const uint8_t *>(prep);
    p.nblk = delta_blocks_per_row(a);
    p.slots = delta_slots(a);
    p.R = (int)(a.nheads / a.ngroups);
    p.nsl = (int)((a.headdim + 63) / 64);
    p.units = (p.R * p.nsl + 1) / 2;
    p.rec = rec ? *rec : dtc::Rec{nullptr, 0, 1};
    const dim3 grid((unsigned)(a.ngroups * p.units), (unsigned)(a.cu_seqlens ? a.nseqs : a.batch));
    const bool dual = p.nsl % 2 != 0;
    if (rec) {
        if (a.dstate <= 64) return dual ? run<64, true, true>(p, grid, m, st) : run<64, false, true>(p, grid, m, st);
        return dual ? run<128, true, true>(p, grid, m, st) : run<128, false, true>(p, grid, m, st);
    }
    if (a.dstate <= 64) return dual ? run<64, true, false>(p, grid, m, st) : run<64, false, false>(p, grid, m, st);
    return dual ? run<128, true, false>(p, grid, m, st) : run<128, false, false>(p, grid, m, st);
}

cudaError_t launch_delta_tc(const ssm_delta_args &a, const SeqView &sv, void *ws, cudaStream_t st) {
    if ((a.cu_seqlens ? a.nseqs : a.batch) == 0) return cudaSuccess;
    DeltaMaps m;
    if (!delta_maps(a, &m)) return cudaErrorInvalidValue;
    cudaError_t e = launch_delta_prep(a, sv, m, ws, false, st);
    if (e != cudaSuccess) return e;
    timing_begin(st);
    e = launch_delta_chain(a, sv, m, ws, nullptr, st);
    timing_end(st);
    return e;
}

}  // namespace ssm
