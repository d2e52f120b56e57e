// delta_prep.cu -- the triangular inverse behind the blocked gated delta rule.
//
// Within a block of 64 tokens, with cs the inclusive prefix sum of the log
// decays and h the state entering the block,
//     u_i = beta_i (v_i - exp(cs_i) h k_i - sum_{j<i} exp(cs_i - cs_j) (k_i . k_j) u_j),
// so U = T R with R_i = beta_i (v_i - exp(cs_i) h k_i), T = (I + M)^-1 and
// M_ij = beta_i exp(cs_i - cs_j) (k_i . k_j) below the diagonal.
//
// One CTA per (block, heads of one group): K K^T once on mma.sync for all the
// heads (bf16 operands are exact, so the products are), then per head M in
// fp32, the four 16 x 16 diagonal blocks by forward substitution (stable
// however alike the keys are, which a series in powers of M is not), and the
// blocks below by T_ij = -T_ii sum_k M_ik T_kj, warp j keeping column j in
// registers: tf32 products with each factor in two parts, about fp32.  T goes
// out as two bf16 parts in the layout the tensor-core kernels read.
#include "delta_tc.cuh"

namespace ssm {
namespace {

using namespace dtc;

constexpr int kLd = 68;                    // row of an fp32 64 x 64 tile

struct PrepArgs {
    const __nv_bfloat16 *k;
    int64_t k_bs, k_ts;
    const float *g, *beta;
    int64_t g_bs, g_ts, b_bs, b_ts;
    const int32_t *cu;
    const int32_t *err;
    int nseqs, H, G, N, heads_per_cta;
    int64_t seqlen, nblk;
    uint8_t *T;                            // [slot][H][kTBytes]
};

struct PrepSmem {
    uint8_t k[2 * kTile];
    float m[kQ * kLd], t[kQ * kLd];
    float hi[kQ], lo[kQ], beta[kQ];
};

SSM_DEVINL void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
SSM_DEVINL void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
SSM_DEVINL void mma1688(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
SSM_DEVINL void tf32_parts(float x, uint32_t &hi, uint32_t &lo) {
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
}

// acc[2 column tiles][4] += A B for 16 x 16 blocks.  A is an accumulator
// fragment (element (g, 8 s + 2 t + e) of k-step s, g = lane / 4, t = lane % 4):
// read as an A fragment its k index t stands for column 2 t and t + 4 for
// 2 t + 1, so B is loaded with its rows in that order.  B[k][n] = b[n][k].
SSM_DEVINL void mul16(float (&acc)[2][4], const float (&a)[2][4], const float *b, int g, int t) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        uint32_t ah[4], al[4];
        tf32_parts(a[s][0], ah[0], al[0]);
        tf32_parts(a[s][2], ah[1], al[1]);
        tf32_parts(a[s][1], ah[2], al[2]);
        tf32_parts(a[s][3], ah[3], al[3]);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float2 v = *reinterpret_cast<const float2 *>(b + (8 * n + g) * kLd + 8 * s + 2 * t);
            uint32_t h0, l0, h1, l1;
            tf32_parts(v.x, h0, l0);
            tf32_parts(v.y, h1, l1);
            mma1688(acc[n], al, h0, h1);
            mma1688(acc[n], ah, l0, l1);
            mma1688(acc[n], ah, h0, h1);
        }
    }
}

template <int NK>
__global__ void __launch_bounds__(128) delta_prep_kernel(const PrepArgs p) {
    if (p.err && *p.err != 0) return;
    extern __shared__ uint8_t raw[];
    PrepSmem &sm = *reinterpret_cast<PrepSmem *>((reinterpret_cast<uintptr_t>(raw) + 127) & ~(uintptr_t)127);
    const Block b = find_block(p.cu, p.nseqs, p.seqlen, p.nblk, blockIdx.x);
    if (b.nt == 0) return;
    const int h0 = blockIdx.y * p.heads_per_cta, R = p.H / p.G, grp = h0 / R;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const __nv_bfloat16 *k = p.k + b.row * p.k_bs + b.t0 * p.k_ts + (int64_t)grp * p.N;
#pragma unroll
    for (int i = tid; i < kQ * NK / 8; i += 128) {
        const int r = i / (NK / 8), c = i % (NK / 8) * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < b.nt && c < p.N) v = *reinterpret_cast<const uint4 *>(k + r * p.k_ts + c);
        *reinterpret_cast<uint4 *>(sm.k + (c >> 6) * kTile + swz(r, c & 63)) = v;
    }
    __syncthreads();
    float kk[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) kk[n][e] = 0.f;
    const uint32_t kb = tc::smem_u32(sm.k);
#pragma unroll
    for (int s = 0; s < NK / 16; ++s) {
        uint32_t a[4];
        const uint32_t at = kb + (s >> 2) * kTile;
        ldsm4(a, at + swz(16 * w + (lane & 15), (s & 3) * 16 + (lane >> 4) * 8));
#pragma unroll
        for (int n2 = 0; n2 < 4; ++n2)
            if (n2 <= w) {
                uint32_t bb[4];
                ldsm4(bb, at + swz(16 * n2 + (lane & 7) + (lane >> 4) * 8, (s & 3) * 16 + ((lane >> 3) & 1) * 8));
                mma16816(kk[2 * n2], a, bb[0], bb[1]);
                mma16816(kk[2 * n2 + 1], a, bb[2], bb[3]);
            }
    }
    for (int hh = 0; hh < p.heads_per_cta; ++hh) {
        const int h = h0 + hh;
        if (w == 0) {
            const float *gp = p.g + b.row * p.g_bs + b.t0 * p.g_ts + h, *bp = p.beta + b.row * p.b_bs + b.t0 * p.b_ts + h;
            const float g0 = lane < b.nt ? fmaxf(gp[lane * p.g_ts], kMinLogDecay) : 0.f;
            const float g1 = lane + 32 < b.nt ? fmaxf(gp[(lane + 32) * p.g_ts], kMinLogDecay) : 0.f;
            double c0, c1, last;
            block_cs(g0, g1, c0, c1, last);
            sm.hi[lane] = (float)c0;
            sm.lo[lane] = (float)(c0 - (double)(float)c0);
            sm.hi[lane + 32] = (float)c1;
            sm.lo[lane + 32] = (float)(c1 - (double)(float)c1);
            sm.beta[lane] = lane < b.nt ? bp[lane * p.b_ts] : 0.f;
            sm.beta[lane + 32] = lane + 32 < b.nt ? bp[(lane + 32) * p.b_ts] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < 8; ++n)
            if (n < 2 * (w + 1)) {
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {
                    const int i = 16 * w + g + 8 * e2, j = 8 * n + 2 * t;
                    float2 v = make_float2(0.f, 0.f);
                    if (j < i && i < b.nt)
                        v.x = sm.beta[i] * ex2(((sm.hi[i] - sm.hi[j]) + (sm.lo[i] - sm.lo[j])) * kLog2e) * kk[n][2 * e2];
                    if (j + 1 < i && i < b.nt)
                        v.y = sm.beta[i] * ex2(((sm.hi[i] - sm.hi[j + 1]) + (sm.lo[i] - sm.lo[j + 1])) * kLog2e) *
                              kk[n][2 * e2 + 1];
                    *reinterpret_cast<float2 *>(sm.m + i * kLd + j) = v;
                }
            }
        __syncthreads();
        {   // column `lane % 16` of the inverse of diagonal block w
            const int c = lane & 15;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s = i == c ? 1.f : 0.f;
                const float *row = sm.m + (16 * w + i) * kLd + 16 * w;
#pragma unroll
                for (int j4 = 0; j4 < i; j4 += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(row + j4);
                    s = fmaf(-v.x, x[j4], s);
                    if (j4 + 1 < i) s = fmaf(-v.y, x[j4 + 1], s);
                    if (j4 + 2 < i) s = fmaf(-v.z, x[j4 + 2], s);
                    if (j4 + 3 < i) s = fmaf(-v.w, x[j4 + 3], s);
                }
                x[i] = s;
            }
            if (lane < 16)
#pragma unroll
                for (int i = 0; i < 16; ++i) sm.t[(16 * w + i) * kLd + 16 * w + c] = x[i];
        }
        __syncthreads();
        {   // the blocks below it: tT[d] = transpose of T block (w + d, w)
            float tT[3][2][4];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    tT[0][s][e] = sm.t[(16 * w + 8 * s + 2 * t + (e & 1)) * kLd + 16 * w + g + 8 * (e >> 1)];
#pragma unroll
            for (int d = 1; d < 4; ++d) {
                const int i = w + d;
                if (i > 3) break;
                float acc[2][4] = {}, out[2][4] = {};
#pragma unroll
                for (int dk = 0; dk < d; ++dk) mul16(acc, tT[dk], sm.m + 16 * i * kLd + 16 * (w + dk), g, t);
                mul16(out, acc, sm.t + 16 * i * kLd + 16 * i, g, t);
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v = -out[s][e];
                        if (d < 3) tT[d][s][e] = v;
                        sm.t[(16 * i + 8 * s + 2 * t + (e & 1)) * kLd + 16 * w + g + 8 * (e >> 1)] = v;
                    }
            }
        }
        __syncthreads();
        uint8_t *out = p.T + ((int64_t)blockIdx.x * p.H + h) * kTBytes;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int i = (tid >> 3) + 16 * it, c = (tid & 7) * 8;
            uint32_t hi[4] = {}, lo[4] = {};
            if (c <= (i | 15))
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 v = *reinterpret_cast<const float2 *>(sm.t + i * kLd + c + 2 * e);
                    split2(v.x, v.y, hi[e], lo[e]);
                }
            *reinterpret_cast<uint4 *>(out + swz(i, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(out + kTile + swz(i, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

}  // namespace

size_t delta_prep_bytes(const ssm_delta_args &a) { return (size_t)delta_slots(a) * a.nheads * kTBytes; }

cudaError_t launch_delta_prep(const ssm_delta_args &a, const SeqView &sv, void *T, cudaStream_t st) {
    PrepArgs p;
    p.k = static_cast<const __nv_bfloat16 *>(a.k);
    p.k_bs = a.k_batch_stride; p.k_ts = a.k_token_stride;
    p.g = a.g; p.beta = a.beta;
    p.g_bs = a.g_batch_stride; p.g_ts = a.g_token_stride;
    p.b_bs = a.beta_batch_stride; p.b_ts = a.beta_token_stride;
    p.cu = a.cu_seqlens; p.err = sv.err; p.nseqs = sv.nseqs;
    p.H = (int)a.nheads; p.G = (int)a.ngroups; p.N = (int)a.dstate;
    p.seqlen = a.seqlen; p.nblk = delta_blocks_per_row(a);
    p.T = static_cast<uint8_t *>(T);
    // as many heads of a group per CTA (they share K K^T) as leave the GPU full
    const int64_t slots = delta_slots(a), R = a.nheads / a.ngroups;
    int hpc = (int)R;
    while (hpc > 1 && (R % hpc != 0 || slots * (a.nheads / hpc) < 8LL * sm_count())) --hpc;
    p.heads_per_cta = hpc;
    const dim3 grid((unsigned)slots, (unsigned)(a.nheads / hpc));
    const size_t smem = sizeof(PrepSmem) + 128;
    auto kernel = a.dstate <= 64 ? delta_prep_kernel<64> : delta_prep_kernel<128>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, 128, smem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace ssm
