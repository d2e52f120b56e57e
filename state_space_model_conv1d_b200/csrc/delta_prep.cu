// delta_prep.cu -- what the blocked gated delta rule needs of every (block,
// head) and what does not depend on the state: the triangular inverse T and
// the attention weights.
//
// Within a block of 64 tokens, with cs the inclusive prefix sum of the log
// decays and h the state entering the block,
//     u_i = beta_i (v_i - exp(cs_i) h k_i - sum_{j<i} exp(cs_i - cs_j) (k_i . k_j) u_j),
// so U = T R with R_i = beta_i (v_i - exp(cs_i) h k_i), T = (I + M)^-1 and
// M_ij = beta_i exp(cs_i - cs_j) (k_i . k_j) below the diagonal; the output
// needs P_ij = scale exp(cs_i - cs_j) (q_i . k_j) up to it.
//
// One CTA per (block, heads of one group), four warps.  [K; Q] K^T is one
// group of tcgen05 MMAs for all the heads and stays in tensor memory, a row in
// each lane.  Then, two heads at a time, warps 2 and 3 make P and warps 0 and
// 1 make M (fp32, shared memory) and invert one head each: lane = column, both
// 32 x 32 diagonal blocks by forward substitution side by side (stable however
// alike the keys are, which a series in powers of M is not), then
// T21 = -T22 (M21 T11).  Rows of M and T22 are read by all lanes at once as 16
// bytes and multiplied two columns at a time.  T goes out as two bf16 parts
// and P as bf16, both in the swizzled layout that the chain's operands have.
// Bound by latency and by shared memory: the inverse reads every row as 16-byte
// broadcasts, four cycles of return bandwidth each.  4 x 4096 tokens, 32 heads in
// 16 groups, N 128 (8192 inverses): 129 us for 134 MB read and 201 MB written;
// 28301 packed tokens, 64 heads of one group (28.8 thousand): 400 us.
#include <string.h>

#include "delta_tc.cuh"
#include "delta_tc.h"

namespace ssm {
namespace {

using namespace dtc;

constexpr int kLd = 68;                    // row of an fp32 64 x 64 tile (16-byte aligned, 4 banks further each row)
constexpr int kPair = 2;                   // heads in work at a time

struct PrepArgs {
    const float *g, *beta;
    int64_t g_bs, g_ts, b_bs, b_ts;
    const int32_t *cu;
    int32_t *err;
    int nseqs, H, G, heads_per_cta;
    int64_t seqlen, nblk;
    float scale;
    uint8_t *out;                          // [slot][H][kHeadBytes or kHeadBytesBwd]
    int bwd;
};

struct Gates {
    float hi[kQ], lo[kQ], beta[kQ];        // prefix sums in two parts
};
struct Head {
    float m[kQ * kLd];                     // M, then T22 in its place and T's high part over the first rows
    uint8_t lo[kTile];                     // T's low part
};
struct PrepSmem {
    union {
        uint8_t kq[4 * kTile];             // per 64-column atom: K rows, Q rows
        Head head[kPair];
    };
    Gates gates[kPair];
    uint64_t full, done;                   // K and Q are here, their products are made: one phase each
    uint32_t tmem;
    int abort;
};

// Bulk copy shared -> global of this warp's own writes (one thread), and the wait until it has read them.
SSM_DEVINL void bulk_store(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(dst), "r"(tc::smem_u32(src)),
                 "r"(bytes)
                 : "memory");
}

// acc = sum over k < 4 n4 of row[k] x[k], two columns at a time.
template <int N4>
SSM_DEVINL float dot_row(const float *row, const float2 *x) {
    float2 a0 = make_float2(0.f, 0.f), a1 = a0;
#pragma unroll
    for (int k = 0; k < N4; ++k) {
        const float4 u = *reinterpret_cast<const float4 *>(row + 4 * k);
        a0 = __ffma2_rn(make_float2(u.x, u.y), x[2 * k], a0);
        a1 = __ffma2_rn(make_float2(u.z, u.w), x[2 * k + 1], a1);
    }
    return (a0.x + a0.y) + (a1.x + a1.y);
}

// The same for two columns x and y at once: a row read from shared memory, whose
// return bandwidth bounds this kernel, serves both.
template <int N4>
SSM_DEVINL float2 dot_row2(const float *row, const float2 *x, const float2 *y) {
    float2 a = make_float2(0.f, 0.f), b = a;
#pragma unroll
    for (int k = 0; k < N4; ++k) {
        const float4 u = *reinterpret_cast<const float4 *>(row + 4 * k);
        a = __ffma2_rn(make_float2(u.x, u.y), x[2 * k], a);
        b = __ffma2_rn(make_float2(u.x, u.y), y[2 * k], b);
        a = __ffma2_rn(make_float2(u.z, u.w), x[2 * k + 1], a);
        b = __ffma2_rn(make_float2(u.z, u.w), y[2 * k + 1], b);
    }
    return make_float2(a.x + a.y, b.x + b.y);
}

// T = (I + M)^-1 of one head, in place, then as two bf16 parts, by two warps
// (`part` 0, 1; they meet at barrier `bar`).  The loops are short on purpose:
// unrolled altogether they would leave the instruction cache.
SSM_DEVINL void invert(Head &hd, int lane, int part, int bar) {
    float *m = hd.m;
    const int c = lane & 15, up = lane >> 4;
    const auto meet = [&] { asm volatile("bar.sync %0, 64;\n" ::"r"(bar) : "memory"); };
    {   // the 32 x 32 diagonal block `part`: its two 16 x 16 blocks (half a warp each, lane = column) by forward
        // substitution; M is zero at and above the diagonal, and so are the x not known yet
        float *d0 = m + 32 * part * (kLd + 1), *d = d0 + 16 * up * (kLd + 1);
        float2 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float2 a0 = make_float2(0.f, 0.f), a1 = a0;
#pragma unroll
            for (int k = 0; k < i; k += 4) {
                const float4 u = *reinterpret_cast<const float4 *>(d + i * kLd + k);
                a0 = __ffma2_rn(make_float2(u.x, u.y), x[k / 2], a0);
                a1 = __ffma2_rn(make_float2(u.z, u.w), x[k / 2 + 1], a1);
            }
            const float v = (i == c ? 1.f : 0.f) - ((a0.x + a0.y) + (a1.x + a1.y));
            if (i & 1) x[i / 2].y = v;
            else x[i / 2].x = v;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) d[i * kLd + c] = i & 1 ? x[i / 2].y : x[i / 2].x;
        __syncwarp();
        // the block below the first: T21 = -T22 (M21 T11), a column of T11 in each lane of half a warp, rows split
        if (up)
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = make_float2(d0[2 * k * kLd + c], d0[(2 * k + 1) * kLd + c]);
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            const float *a = d0 + 16 * kLd + (pass ? 16 : 0);
            float z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = dot_row<4>(a + (8 * up + i) * kLd, x);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) d0[(16 + 8 * up + i) * kLd + c] = pass ? -z[i] : z[i];
            __syncwarp();
            if (pass == 0)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    x[k] = make_float2(d0[(16 + 2 * k) * kLd + c], d0[(17 + 2 * k) * kLd + c]);
        }
    }
    meet();
    // the 32 x 32 block below: 16 rows per warp, 8 per half warp; columns 2 c and 2 c + 1 in each lane
    float2 x[16], y[16];
    const auto at2 = [&](int row, int col) -> float2 & { return *reinterpret_cast<float2 *>(m + row * kLd + col); };
    const auto columns = [&](int row) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float2 u = at2(row + 2 * k, 2 * c), v = at2(row + 2 * k + 1, 2 * c);
            x[k] = make_float2(u.x, v.x);
            y[k] = make_float2(u.y, v.y);
        }
    };
    columns(0);
    const int r0 = 32 + 16 * part + 8 * up;
#pragma unroll 1
    for (int i = r0; i < r0 + 8; i += 2) {
        const float2 z0 = dot_row2<8>(m + i * kLd, x, y), z1 = dot_row2<8>(m + (i + 1) * kLd, x, y);
        __syncwarp();
        at2(i, 2 * c) = z0;
        at2(i + 1, 2 * c) = z1;
    }
    // The high part of T lies over the fp32 rows: row i of it ends at byte 128 (i + 1), row j of those begins at
    // 272 j, so T's rows 0 - 31 (first warp, in order) only meet fp32 rows that are read, and rows 32 - 63 end
    // before fp32 row 32.
    uint8_t *hi = reinterpret_cast<uint8_t *>(m), *lo = hd.lo;
    const auto word = [](uint8_t *t, int i, int j) -> uint32_t & { return *reinterpret_cast<uint32_t *>(t + swz(i, j)); };
    if (part == 1 && lane == 0) tc::bulk_wait_read();  // the attention weights have left the low part's place
    meet();                                            // the products are written, T11 is read
    columns(32);
    const int t0 = 32 * part;                          // first warp: T11; second: T22's low part, T22 itself stays
#pragma unroll 1
    for (int i = 0; i < 32; i += 8) {
        float2 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = at2(t0 + i + 2 * e + up, t0 + 2 * c);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = i + 2 * e + up;
            uint32_t h, l;
            split2(v[e].x, v[e].y, h, l);
            word(lo, t0 + row, t0 + 2 * c) = l;
            if (part == 0) {
                word(hi, row, 2 * c) = h;
                word(hi, row, 32 + 2 * c) = 0;
                word(lo, row, 32 + 2 * c) = 0;
            }
        }
    }
    meet();                                            // T11's fp32 rows are read
#pragma unroll 1
    for (int i = r0; i < r0 + 8; i += 2) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // T22's rows 0 - 15 end at column 16
            const float *t = m + (i + e) * kLd + 32;
            const float2 z = part == 0 ? dot_row2<4>(t, x, y) : dot_row2<8>(t, x, y), v = at2(i + e, 32 + 2 * c);
            uint32_t h, l;
            split2(-z.x, -z.y, h, l);
            word(hi, i + e, 2 * c) = h;
            word(lo, i + e, 2 * c) = l;
            word(hi, i + e, 32 + 2 * c) = pack2(v.x, v.y);
        }
    }
    tc::fence_proxy_async();
    meet();
}

template <int NK>
__global__ void __launch_bounds__(128, 4) delta_prep_kernel(const PrepArgs p, const __grid_constant__ CUtensorMap tm_q,
                                                               const __grid_constant__ CUtensorMap tm_k) {
    if (p.err && *p.err != 0) return;
    extern __shared__ uint8_t raw[];
    PrepSmem &sm = *reinterpret_cast<PrepSmem *>(smem_1024(raw));
    const Block b = find_block(p.cu, p.nseqs, p.seqlen, p.nblk, blockIdx.x);
    if (b.nt == 0) return;
    const int h0 = blockIdx.y * p.heads_per_cta, R = p.H / p.G, grp = h0 / R;
    if (!SSM_BOUNDS(b.s, p.nseqs, BS_DELTA_SEQ) || !SSM_BOUNDS(b.t0 + b.nt - 1, p.seqlen, BS_DELTA_SEQ) ||
        !SSM_BOUNDS(seq_slot(p.cu, b.s, p.nblk) + (b.t0 - (p.cu ? p.cu[b.s] : 0)) / kQ - blockIdx.x, 1, BS_DELTA_SLOT) ||
        !SSM_BOUNDS(h0 + p.heads_per_cta - 1, p.H, BS_DELTA_HEAD)) return;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    if (w == 0) tc::tmem_alloc(&sm.tmem, 64);
    if (tid == 0) {
        tc::mbar_init(&sm.full, 1);
        tc::mbar_init(&sm.done, 1);
        tc::mbar_init_fence();
        sm.abort = 0;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = sm.tmem;
    bool ok = true;
    if (tid == 0) {
        // rows behind the sequence's end may hold anything: a product only meets its own two rows
        tc::mbar_expect_tx(&sm.full, NK / 64 * 2 * kTile);
#pragma unroll
        for (int x = 0; x < NK / 64; ++x) {
            tma_load_4d(sm.kq + x * 2 * kTile, &tm_k, 64 * x, grp, (int)b.t0, (int)b.row, &sm.full);
            tma_load_4d(sm.kq + x * 2 * kTile + kTile, &tm_q, 64 * x, grp, (int)b.t0, (int)b.row, &sm.full);
        }
        ok = wait_bar(&sm.full, &sm.abort, 0, p.err) || tc::mbar_wait(&sm.full, 0, 1u << 22);
        tc::fence_after_sync();
        const uint64_t d = tc::desc_sw128(tc::smem_u32(sm.kq), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < NK / 16; ++kk) {
            const uint32_t o = ((kk >> 2) * 2 * kTile + (kk & 3) * 32) >> 4;
            tc::mma_bf16(tm, d + o, d + o, tc::idesc_bf16(128, 64, 0, 0), kk > 0);
        }
        tc::mma_commit(&sm.done);
    }
    __syncwarp();
    const uint32_t tl = tm + ((uint32_t)(32 * w) << 16);
    const int64_t hbytes = p.bwd ? kHeadBytesBwd : kHeadBytes;
    const int i = (w & 1) * 32 + lane;                 // this thread's row of K K^T (warps 0, 1) or Q K^T (2, 3)
    for (int hb = 0; hb < p.heads_per_cta; hb += kPair) {
        const int nh = min(kPair, p.heads_per_cta - hb);
        if (w >= 2 && w - 2 < nh) {
            Gates &gt = sm.gates[w - 2];
            const int h = h0 + hb + w - 2;
            const float *gp = p.g + b.row * p.g_bs + b.t0 * p.g_ts + h, *bp = p.beta + b.row * p.b_bs + b.t0 * p.b_ts + h;
            const float g0 = lane < b.nt ? log_decay(gp[lane * p.g_ts]) : 0.f;
            const float g1 = lane + 32 < b.nt ? log_decay(gp[(lane + 32) * p.g_ts]) : 0.f;
            float b0 = lane < b.nt ? bp[lane * p.b_ts] : 0.f, b1 = lane + 32 < b.nt ? bp[(lane + 32) * p.b_ts] : 0.f;
            if (p.bwd) {
                b0 = bwd_beta(b0);
                b1 = bwd_beta(b1);
            }
            double c0, c1, last;
            block_cs(g0, g1, c0, c1, last);
            gt.hi[lane] = (float)c0;
            gt.lo[lane] = (float)(c0 - (double)(float)c0);
            gt.hi[lane + 32] = (float)c1;
            gt.lo[lane + 32] = (float)(c1 - (double)(float)c1);
            gt.beta[lane] = b0;
            gt.beta[lane + 32] = b1;
        }
        if (hb == 0) {                                 // the products were made meanwhile
            // (after a wait that ran out, one more of a fixed length: what is in flight lands before the CTA ends)
            ok = (wait_bar(&sm.done, &sm.abort, 0, p.err) || tc::mbar_wait(&sm.done, 0, 1u << 22)) && ok && !sm.abort;
            tc::fence_after_sync();
        }
        if (!__syncthreads_and(ok)) break;             // (the error word is set; nothing was computed)
        for (int hh = 0; hh < nh; ++hh) {
            const Gates &gt = sm.gates[hh];
            const float ch = gt.hi[i], cl = gt.lo[i];
            uint8_t *out = p.out + ((int64_t)blockIdx.x * p.H + h0 + hb + hh) * hbytes;
            if (w < 2) {
                const float be = i < b.nt ? gt.beta[i] : 0.f;
                float *row = sm.head[hh].m + i * kLd;
#pragma unroll 1
                for (int c = 0; c <= w; ++c) {         // (columns 32-63 of rows 0-31 are not read)
                    float v[32];
                    tc::tmem_ld32(tl + 32 * c, v);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 jh = *reinterpret_cast<const float4 *>(gt.hi + 32 * c + e);
                        const float4 jl = *reinterpret_cast<const float4 *>(gt.lo + 32 * c + e);
                        const float dh[4] = {jh.x, jh.y, jh.z, jh.w}, dl[4] = {jl.x, jl.y, jl.z, jl.w};
                        float o[4];
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            o[f] = 32 * c + e + f < i && i < b.nt
                                       ? be * ex2(((ch - dh[f]) + (cl - dl[f])) * kLog2e) * v[e + f] : 0.f;
                        *reinterpret_cast<float4 *>(row + 32 * c + e) = make_float4(o[0], o[1], o[2], o[3]);
                    }
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    float v[32];
                    if (c <= w - 2) tc::tmem_ld32(tl + 32 * c, v);
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t o[4] = {0, 0, 0, 0}, ol[4] = {0, 0, 0, 0};
                        if (c <= w - 2 && i < b.nt)
#pragma unroll
                            for (int f = 0; f < 4; ++f) {
                                const int j = 32 * c + e + 2 * f;
                                const float2 cj = *reinterpret_cast<const float2 *>(gt.hi + j);
                                const float2 lj = *reinterpret_cast<const float2 *>(gt.lo + j);
                                const float e0 = ex2(((ch - cj.x) + (cl - lj.x)) * kLog2e);
                                const float e1 = ex2(((ch - cj.y) + (cl - lj.y)) * kLog2e);
                                const float v0 = j <= i ? e0 * (v[e + 2 * f] * p.scale) : 0.f;
                                const float v1 = j < i ? e1 * (v[e + 2 * f + 1] * p.scale) : 0.f;
                                split2(v0, v1, o[f], ol[f]);
                            }
                        // by way of T's low part's place: a lane's own row of 128 bytes would take a line per store
                        *reinterpret_cast<uint4 *>(sm.head[hh].lo + swz(i, 32 * c + e)) = make_uint4(o[0], o[1], o[2], o[3]);
                        if (p.bwd)
                            *reinterpret_cast<uint4 *>(out + kTBytes + kTile + swz(i, 32 * c + e)) =
                                make_uint4(ol[0], ol[1], ol[2], ol[3]);
                    }
                }
            }
        }
        tc::fence_proxy_async();
        __syncthreads();                               // M and P are written
        if ((w & 1) < nh) {
            Head &hd = sm.head[w & 1];
            if (w >= 2 && lane == 0) {
                bulk_store(p.out + ((int64_t)blockIdx.x * p.H + h0 + hb + w - 2) * hbytes + kTBytes, hd.lo, kTile);
                asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
            }
            invert(hd, lane, w >> 1, 2 + (w & 1));
            if (tid < 64 && lane == 0) {
                uint8_t *out = p.out + ((int64_t)blockIdx.x * p.H + h0 + hb + w) * hbytes;
                bulk_store(out, hd.m, kTile);
                bulk_store(out + kTile, hd.lo, kTile);
                asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
                tc::bulk_wait_read();                  // the tile may be overwritten, or the CTA end
            }
        }
        __syncthreads();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (w == 0) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tm, 64);
    }
}

}  // namespace

size_t delta_prep_bytes(const ssm_delta_args &a, bool bwd) {
    return (size_t)delta_slots(a) * a.nheads * (bwd ? dtc::kHeadBytesBwd : dtc::kHeadBytes);
}

cudaError_t launch_delta_prep(const ssm_delta_args &a, const SeqView &sv, const DeltaMaps &m, void *out, bool bwd,
                              cudaStream_t st) {
    PrepArgs p;
    p.g = a.g; p.beta = a.beta;
    p.g_bs = a.g_batch_stride; p.g_ts = a.g_token_stride;
    p.b_bs = a.beta_batch_stride; p.b_ts = a.beta_token_stride;
    p.cu = a.cu_seqlens; p.err = sv.err; p.nseqs = sv.nseqs;
    p.H = (int)a.nheads; p.G = (int)a.ngroups;
    p.seqlen = a.seqlen; p.nblk = delta_blocks_per_row(a);
    p.scale = a.scale;
    p.out = static_cast<uint8_t *>(out);
    p.bwd = bwd;
    // as many heads of a group per CTA (they share [K; Q] K^T) as leave the GPU full.  The whole forward in us with
    // this rule / one head / all heads a CTA: 16 x 2048 tokens, 64 heads of one group 1001 / 1227 / 1044,
    // 4 x 4096, 32 of 16 groups 381 / 431 / 381, 1 x 512, 32 of one 58 / 58 / 184
    const int64_t slots = delta_slots(a), R = a.nheads / a.ngroups;
    int hpc = (int)R;
    while (hpc > 1 && (R % hpc != 0 || slots * (a.nheads / hpc) < 16LL * sm_count())) --hpc;
    p.heads_per_cta = hpc;
    const dim3 grid((unsigned)slots, (unsigned)(a.nheads / hpc));
    const size_t smem = sizeof(PrepSmem) + 1024;
    auto kernel = a.dstate <= 64 ? delta_prep_kernel<64> : delta_prep_kernel<128>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, 128, smem, st>>>(p, m.q, m.k);
    return cudaGetLastError();
}

}  // namespace ssm
