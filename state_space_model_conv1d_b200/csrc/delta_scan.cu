// delta_scan.cu -- the gated delta rule token by token in fp32 (any dtype and
// sizes), forward and backward.
//
// A state row h[p, :] never meets another one:
//     w = a_t h,  s = w . k_t,  u = beta_t (v_t[p] - s),  h = w + u k_t,
//     y_t[p] = scale (h . q_t) = scale (w . q_t + u (k_t . q_t)),
// so rows are spread over lanes: 8 lanes hold one row (4 consecutive states
// of every 32) and a warp 4 rows, or 16 or 32 lanes a row where rows are few.
// The dot product that the chain waits for is summed in one pass of shuffles.
// The chain over the tokens bounds the time (about 170 ns a token), not memory;
// a sequence's rows run in separate CTAs.  2 x 333 tokens, 6 heads, P 40, N 72,
// fp32: 57 us (2.7 MB, 0.4 us of HBM); the gradients of 5 packed sequences of
// 517 tokens, 4 heads, P 48, N 64: 32 us for the checkpoints, 115 us backwards
// and 6 us for the sums.
//
// Backward, per row, from the last token to the first, with d = dL/dh_t:
//     d += scale dy q;  du = d . k;  dv = beta du;  ds = -beta du;
//     dbeta = sum_p du (v - s);  dq = scale sum_p dy h_t;
//     dk = sum_p (u d + ds w);  d += ds k;  dg = sum_{p,n} d w;  d = a d.
// The states before every 32nd token are kept by a forward pass; the tokens
// between are recomputed, in runs that fit in registers or, with few rows, once
// into shared memory.  Each CTA owns some rows and writes their share of dq,
// dk, dg, dbeta; a last kernel adds the shares in a fixed order.
#include "common.cuh"
#include "delta.h"

namespace ssm {
namespace {

// L lanes per state row, W warps per CTA.
template <int L, int W> struct Cut {
    static constexpr int threads = W * 32, rows = W * 32 / L, per_warp = 32 / L;
};

struct Args {
    ssm_delta_args a;
    SeqView sv;
    float *ckpt;
    int64_t ckpt_rows;
};

// Tokens [lo, hi) of the sequence this CTA owns; row = batch row.
struct Seq {
    int s;
    int64_t row, lo, hi, ckpt_row;
};
SSM_DEVINL Seq find_seq(const ssm_delta_args &a, const SeqView &sv, int y) {
    Seq q;
    if (a.cu_seqlens) {
        q.s = sv.order[y];
        q.row = 0;
        q.lo = a.cu_seqlens[q.s];
        q.hi = a.cu_seqlens[q.s + 1];
        q.ckpt_row = q.lo / kDeltaCkpt + q.s;
    } else {
        q.s = y;
        q.row = y;
        q.lo = 0;
        q.hi = a.seqlen;
        q.ckpt_row = (int64_t)y * ((a.seqlen + kDeltaCkpt - 1) / kDeltaCkpt);
    }
    return q;
}

// State index of element e of a row's lane: 4 consecutive of every 4 L.
template <int L> SSM_DEVINL int state_of(int lrow, int e) { return (e >> 2) * 4 * L + lrow * 4 + (e & 3); }

// `nt` tokens of a [tokens][width] operand on the way to shared memory, fp32,
// PAD columns wide (zeros past width and behind nt): all of a thread's loads
// are issued together, while the tokens before are still in work.
template <typename T, int PAD, int kTok, int kThreads> struct Staged {
    static constexpr int kPer = kTok * PAD / kThreads;
    float v[kPer];
    SSM_DEVINL void load(const T *src, int64_t ts, int nt, int width) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            // (token and column without a division wherever one count divides the other)
            int t, c;
            if constexpr (PAD % kThreads == 0) {
                t = i * kThreads / PAD;
                c = threadIdx.x + i * kThreads % PAD;
            } else if constexpr (kThreads % PAD == 0) {
                t = threadIdx.x / PAD + i * (kThreads / PAD);
                c = threadIdx.x % PAD;
            } else {
                const int x = threadIdx.x + i * kThreads;
                t = x / PAD;
                c = x % PAD;
            }
            v[i] = (t < nt && c < width) ? Elem<T>::ld(src + (int64_t)t * ts + c) : 0.f;
        }
    }
    SSM_DEVINL void store(float *dst) const {
#pragma unroll
        for (int i = 0; i < kPer; ++i) dst[threadIdx.x + i * kThreads] = v[i];
    }
};

template <int NE, int L>
SSM_DEVINL void load_row(float (&h)[NE], const float *src, int lrow, int64_t N) {
#pragma unroll
    for (int e = 0; e < NE; ++e) {
        const int n = state_of<L>(lrow, e);
        h[e] = n < N ? src[n] : 0.f;
    }
}
// Sum over a row's lanes.
template <int L> SSM_DEVINL float row_sum(float v) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Y: y is wanted (the checkpoints alone otherwise).  Only the sum that the chain
// waits for is taken at once; y's partial sums, one per lane and token, go to a
// tile of the warp's own and are added after kTok tokens, a token in each lane.
template <int NE, int L, int W, bool Y> constexpr int scan_floats() {
    return (Y ? 2 : 1) * kDeltaCkpt * NE * L + kDeltaCkpt * (Cut<L, W>::rows + 2) + (Y ? W * 32 * 33 : 0);
}
template <typename T, int NE, int L, int W, bool Y>
__global__ void __launch_bounds__(W * 32) delta_scan_kernel(const Args p) {
    constexpr int kThreads = Cut<L, W>::threads, kRows = Cut<L, W>::rows, kTok = kDeltaCkpt;   // tokens staged at a time
    const ssm_delta_args &a = p.a;
    if (p.sv.err && *p.sv.err != 0) return;
    constexpr int NP = NE * L;
    extern __shared__ float sm[];
    float *ks = sm, *qs = ks + kTok * NP, *vs = Y ? qs + kTok * NP : qs, *as = vs + kTok * kRows, *bs = as + kTok;
    const Seq sq = find_seq(a, p.sv, blockIdx.y);
    const int64_t H = a.nheads, P = a.headdim, N = a.dstate;
    const int h = blockIdx.x % H, p0 = (int)(blockIdx.x / H) * kRows;
    const int grp = (int)(h / (H / a.ngroups));
    if (!SSM_BOUNDS(sq.hi, a.seqlen + 1, BS_DELTA_SEQ) || !SSM_BOUNDS(sq.lo, sq.hi + 1, BS_DELTA_SEQ)) return;
    if (p.ckpt && !SSM_BOUNDS(sq.ckpt_row + (sq.hi - sq.lo + kTok - 1) / kTok, p.ckpt_rows + 1, BS_DELTA_CKPT)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lrow = lane % L;
    const int r = warp * Cut<L, W>::per_warp + lane / L;       // row within the CTA
    const bool live = p0 + r < P;
    const int64_t srow = ((int64_t)sq.s * H + h) * P + p0 + r;
    float2 st2[NE / 2];
    {
        float st[NE];
        if (live && a.h0) load_row<NE, L>(st, a.h0 + srow * N, lrow, N);
        else
#pragma unroll
            for (int e = 0; e < NE; ++e) st[e] = 0.f;
#pragma unroll
        for (int e = 0; e < NE / 2; ++e) st2[e] = make_float2(st[2 * e], st[2 * e + 1]);
    }
    const auto keep = [&](float *o) {
#pragma unroll
        for (int e = 0; e < NE; ++e)
            if (state_of<L>(lrow, e) < N) o[state_of<L>(lrow, e)] = e & 1 ? st2[e / 2].y : st2[e / 2].x;
    };

    const T *q = (const T *)a.q + sq.row * a.q_batch_stride + grp * N;
    const T *k = (const T *)a.k + sq.row * a.k_batch_stride + grp * N;
    const T *v = (const T *)a.v + sq.row * a.v_batch_stride + h * P + p0;
    const float *g = a.g + sq.row * a.g_batch_stride + h, *be = a.beta + sq.row * a.beta_batch_stride + h;
    T *y = Y ? (T *)a.y + sq.row * a.y_batch_stride + h * P + p0 + warp * Cut<L, W>::per_warp : nullptr;
    float *ys = bs + kTok + warp * 32 * 33;            // [token][lane]
    const int vw = (int)min((int64_t)kRows, P - p0);
    Staged<T, NP, kTok, kThreads> sk_, sq_s;
    Staged<T, kRows, kTok, kThreads> sv_;
    float ga = 1.f, gb = 0.f;
    const auto fetch = [&](int64_t t0) {
        const int nt = (int)min((int64_t)kTok, sq.hi - t0);
        sk_.load(k + t0 * a.k_token_stride, a.k_token_stride, nt, (int)N);
        if constexpr (Y) sq_s.load(q + t0 * a.q_token_stride, a.q_token_stride, nt, (int)N);
        sv_.load(v + t0 * a.v_token_stride, a.v_token_stride, nt, vw);
        if (threadIdx.x < kTok) {
            const int t = threadIdx.x;
            ga = t < nt ? g[(t0 + t) * a.g_token_stride] : 0.f;
            gb = t < nt ? be[(t0 + t) * a.beta_token_stride] : 0.f;
        }
    };
    if (sq.lo < sq.hi) fetch(sq.lo);
    for (int64_t t0 = sq.lo; t0 < sq.hi; t0 += kTok) {
        const int nt = (int)min((int64_t)kTok, sq.hi - t0);
        if (p.ckpt && live)
            keep(p.ckpt + (((sq.ckpt_row + (t0 - sq.lo) / kDeltaCkpt) * H + h) * P + p0 + r) * N);
        __syncthreads();                               // the tokens before are read
        sk_.store(ks);
        if constexpr (Y) sq_s.store(qs);
        sv_.store(vs);
        if (threadIdx.x < kTok) {
            as[threadIdx.x] = decay_of(ga);
            bs[threadIdx.x] = gb;
        }
        __syncthreads();
        if (t0 + kTok < sq.hi) fetch(t0 + kTok);
        // the next token's operands are on their way while this one's sum runs
        float2 kk[NE / 2], qq[NE / 2];
        float at, bt, vt;
        const auto pairs = [&](float2(&x)[NE / 2], const float *row) {
#pragma unroll
            for (int e = 0; e < NE / 4; ++e) {
                const float4 u = *reinterpret_cast<const float4 *>(row + state_of<L>(lrow, 4 * e));
                x[2 * e] = make_float2(u.x, u.y);
                x[2 * e + 1] = make_float2(u.z, u.w);
            }
        };
        const auto token = [&](int t) {
            pairs(kk, ks + t * NP);
            at = as[t];
            bt = bs[t];
            vt = vs[t * kRows + r];
        };
        const auto part = [](const float2(&x)[2]) { return (x[0].x + x[0].y) + (x[1].x + x[1].y); };
        token(0);
        for (int t = 0; t < nt; ++t) {
            // packed pairs of states, two chains a sum
            const float2 al = make_float2(at, at), zero = make_float2(0.f, 0.f);
            float2 sk2[2] = {zero, zero}, k0[NE / 2];
#pragma unroll
            for (int e = 0; e < NE / 2; ++e) {
                k0[e] = kk[e];
                st2[e] = __fmul2_rn(st2[e], al);
                sk2[e & 1] = __ffma2_rn(st2[e], kk[e], sk2[e & 1]);
            }
            const float b0 = bt, v0 = vt;
            if constexpr (Y) pairs(qq, qs + t * NP);
            token(min(t + 1, kTok - 1));
            const float u = b0 * (v0 - row_sum<L>(part(sk2)));
#pragma unroll
            for (int e = 0; e < NE / 2; ++e) st2[e] = __ffma2_rn(make_float2(u, u), k0[e], st2[e]);
            if constexpr (Y) {
                float2 sy[2] = {zero, zero};
#pragma unroll
                for (int e = 0; e < NE / 2; ++e) sy[e & 1] = __ffma2_rn(st2[e], qq[e], sy[e & 1]);
                ys[t * 33 + lane] = part(sy);
            }
        }
        if constexpr (Y) {
            __syncwarp();
            if (lane < nt)
#pragma unroll
                for (int i = 0; i < Cut<L, W>::per_warp; ++i) {
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int e = 0; e < L; e += 2) {
                        s0 += ys[lane * 33 + i * L + e];
                        s1 += ys[lane * 33 + i * L + e + 1];
                    }
                    if (p0 + warp * Cut<L, W>::per_warp + i < P)
                        Elem<T>::st(y + (t0 + lane) * a.y_token_stride + i, a.scale * (s0 + s1));
                }
            __syncwarp();
        }
    }
    if (a.h_final && live) keep(a.h_final + srow * N);
}

// ------------------------------------------------------------------ backward
struct BwdArgs {
    ssm_delta_bwd_args b;
    SeqView sv;
    const float *ckpt;
    float *pq, *pk;        // [slices][tokens][H][N]
    float *pg, *pb;        // [slices][tokens][H]
    int64_t ckpt_rows, slices;
};

// Sum over the rows of a warp.  With 4 rows lane group i (lanes 8 i .. 8 i + 7)
// ends with a quarter of the elements, those from first_of() on; with one row
// there is nothing to add.
template <int NE, int L> constexpr int kept() { return L == 32 ? NE : NE / 4; }
template <int NE, int L> SSM_DEVINL int first_of(int lane) {
    return L == 32 ? 0 : (((lane >> 4) & 1) * 2 + ((lane >> 3) & 1)) * (NE / 4);
}
template <int NE, int L>
SSM_DEVINL void rows_sum(float (&x)[NE], float (&out)[kept<NE, L>()], int lane) {
    if constexpr (L == 32) {
#pragma unroll
        for (int e = 0; e < NE; ++e) out[e] = x[e];
    } else {
        const bool hi = lane & 16, hi2 = lane & 8;
        float y[NE / 2];
#pragma unroll
        for (int e = 0; e < NE / 2; ++e) {
            const float give = hi ? x[e] : x[e + NE / 2], keep = hi ? x[e + NE / 2] : x[e];
            y[e] = keep + __shfl_xor_sync(~0u, give, 16);
        }
#pragma unroll
        for (int e = 0; e < NE / 4; ++e) {
            const float give = hi2 ? y[e] : y[e + NE / 4], keep = hi2 ? y[e + NE / 4] : y[e];
            out[e] = keep + __shfl_xor_sync(~0u, give, 8);
        }
    }
}

// TR tokens are held in registers at a time (TR * NE states each).
template <typename T, int NE, int TR, int L, int W>
__global__ void __launch_bounds__(W * 32, 1) delta_scan_bwd_kernel(const BwdArgs p) {
    constexpr int kThreads = Cut<L, W>::threads, kRows = Cut<L, W>::rows, kTok = kDeltaCkpt, kWarps = W;
    const ssm_delta_args &a = p.b.fwd;
    if (p.sv.err && *p.sv.err != 0) return;
    constexpr int NP = NE * L;
    extern __shared__ float sm[];
    float *ks = sm, *qs = ks + kTok * NP, *vs = qs + kTok * NP, *ds_ = vs + kTok * kRows, *as = ds_ + kTok * kRows,
          *bs = as + kTok;
    float *rq = bs + kTok;                     // [TR][kWarps][NP] each
    float *rk = rq + TR * kWarps * NP;
    float *rg = rk + TR * kWarps * NP;         // [TR][kWarps]
    float *rb = rg + TR * kWarps;
    const Seq sq = find_seq(a, p.sv, blockIdx.y);
    const int64_t H = a.nheads, P = a.headdim, N = a.dstate;
    const int h = blockIdx.x % H, slice = (int)(blockIdx.x / H), p0 = slice * kRows;
    const int grp = (int)(h / (H / a.ngroups));
    if (!SSM_BOUNDS(sq.hi, a.seqlen + 1, BS_DELTA_SEQ) || !SSM_BOUNDS(sq.lo, sq.hi + 1, BS_DELTA_SEQ)) return;
    if (!SSM_BOUNDS(sq.ckpt_row + (sq.hi - sq.lo + kTok - 1) / kTok, p.ckpt_rows + 1, BS_DELTA_CKPT) ||
        !SSM_BOUNDS(p0, P, BS_DELTA_STATE) || !SSM_BOUNDS(slice, p.slices, BS_DELTA_SHARE)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lrow = lane % L;
    const int r = warp * Cut<L, W>::per_warp + lane / L;
    const bool live = p0 + r < P;
    const int64_t srow = ((int64_t)sq.s * H + h) * P + p0 + r;
    float d[NE];
    if (live && p.b.dh_final) load_row<NE, L>(d, p.b.dh_final + srow * N, lrow, N);
    else
#pragma unroll
        for (int e = 0; e < NE; ++e) d[e] = 0.f;
    const T *q = (const T *)a.q + sq.row * a.q_batch_stride + grp * N;
    const T *k = (const T *)a.k + sq.row * a.k_batch_stride + grp * N;
    const T *v = (const T *)a.v + sq.row * a.v_batch_stride + h * P + p0;
    const T *dy = (const T *)p.b.dy + sq.row * p.b.dy_batch_stride + h * P + p0;
    const float *g = a.g + sq.row * a.g_batch_stride + h, *be = a.beta + sq.row * a.beta_batch_stride + h;
    const int64_t tok0 = sq.row * a.seqlen;    // tokens of all rows are numbered through in the outputs
    const int64_t ntok = a.batch * a.seqlen;
    T *dv = (T *)p.b.dv + h * P + p0;
    const int vw = (int)min((int64_t)kRows, P - p0);

    const int64_t len = sq.hi - sq.lo;
    for (int64_t c = (len + kTok - 1) / kTok - 1; c >= 0; --c) {
        const int64_t t0 = sq.lo + c * kTok;
        const int nt = (int)min((int64_t)kTok, sq.hi - t0);
        __syncthreads();
        {
            Staged<T, NP, kTok, kThreads> s;
            s.load(k + t0 * a.k_token_stride, a.k_token_stride, nt, (int)N);
            Staged<T, kRows, kTok, kThreads> s2, s3;
            s2.load(v + t0 * a.v_token_stride, a.v_token_stride, nt, vw);
            s3.load(dy + t0 * p.b.dy_token_stride, p.b.dy_token_stride, nt, vw);
            s.store(ks);
            s2.store(vs);
            s3.store(ds_);
            s.load(q + t0 * a.q_token_stride, a.q_token_stride, nt, (int)N);
            s.store(qs);
        }
        if (threadIdx.x < kTok) {
            const int t = threadIdx.x;
            as[t] = t < nt ? decay_of(g[(t0 + t) * a.g_token_stride]) : 1.f;
            bs[t] = t < nt ? be[(t0 + t) * a.beta_token_stride] : 0.f;
        }
        __syncthreads();
        const float *cp = p.ckpt + (((sq.ckpt_row + c) * H + h) * P + p0 + r) * N;
        for (int run = (nt + TR - 1) / TR - 1; run >= 0; --run) {
            float st[NE];
            if (live) load_row<NE, L>(st, cp, lrow, N);
            else
#pragma unroll
                for (int e = 0; e < NE; ++e) st[e] = 0.f;
            // forward to the run's first token
            {
                float kn[NE];
#pragma unroll
                for (int e = 0; e < NE; ++e) kn[e] = ks[state_of<L>(lrow, e)];
                for (int t = 0; t < run * TR; ++t) {
                    float sk = 0.f, kt[NE];
                    const float at = as[t];
#pragma unroll
                    for (int e = 0; e < NE; ++e) {
                        kt[e] = kn[e];
                        st[e] *= at;
                        sk = fmaf(st[e], kt[e], sk);
                        kn[e] = ks[(t + 1) * NP + state_of<L>(lrow, e)];       // t + 1 < kTok
                    }
                    const float u = bs[t] * (vs[t * kRows + r] - row_sum<L>(sk));
#pragma unroll
                    for (int e = 0; e < NE; ++e) st[e] = fmaf(u, kt[e], st[e]);
                }
            }
            // through the run: w = a h_{t-1} of every token stays in registers
            float w[TR][NE], uu[TR], sk_[TR];
#pragma unroll
            for (int i = 0; i < TR; ++i) {
                const int t = run * TR + i;                    // t < kTok; tokens behind nt have a = 1, beta = 0
                float sk = 0.f;
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    w[i][e] = st[e] * as[t];
                    sk = fmaf(w[i][e], ks[t * NP + state_of<L>(lrow, e)], sk);
                }
                sk_[i] = row_sum<L>(sk);
                uu[i] = bs[t] * (vs[t * kRows + r] - sk_[i]);
#pragma unroll
                for (int e = 0; e < NE; ++e) st[e] = fmaf(uu[i], ks[t * NP + state_of<L>(lrow, e)], w[i][e]);
            }
#pragma unroll
            for (int i = TR - 1; i >= 0; --i) {
                const int t = run * TR + i;
                const float dyv = a.scale * ds_[t * kRows + r];
                float x[NE], part[kept<NE, L>()], du = 0.f;
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    const int n = t * NP + state_of<L>(lrow, e);
                    x[e] = dyv * fmaf(uu[i], ks[n], w[i][e]);          // dq: dy h_t
                    d[e] = fmaf(dyv, qs[n], d[e]);
                    du = fmaf(d[e], ks[n], du);
                }
                du = row_sum<L>(du);
                rows_sum<NE, L>(x, part, lane);
                const int e0 = first_of<NE, L>(lane);
#pragma unroll
                for (int e = 0; e < kept<NE, L>(); ++e) rq[(i * kWarps + warp) * NP + state_of<L>(lrow, e0 + e)] = part[e];
                const float dsv = -bs[t] * du;
                float dg = 0.f;
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    const int n = t * NP + state_of<L>(lrow, e);
                    x[e] = fmaf(uu[i], d[e], dsv * w[i][e]);
                    d[e] = fmaf(dsv, ks[n], d[e]);
                    dg = fmaf(d[e], w[i][e], dg);
                    d[e] *= as[t];
                }
                rows_sum<NE, L>(x, part, lane);
#pragma unroll
                for (int e = 0; e < kept<NE, L>(); ++e) rk[(i * kWarps + warp) * NP + state_of<L>(lrow, e0 + e)] = part[e];
                float db = lrow == 0 ? du * (vs[t * kRows + r] - sk_[i]) : 0.f;
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    dg += __shfl_xor_sync(~0u, dg, o);
                    db += __shfl_xor_sync(~0u, db, o);
                }
                if (lane == 0) {
                    rg[i * kWarps + warp] = dg;
                    rb[i * kWarps + warp] = db;
                }
                if (lrow == 0 && live && t < nt)
                    Elem<T>::st(dv + (tok0 + t0 + t) * H * P + r, -dsv);
            }
            __syncthreads();
            for (int i = threadIdx.x; i < TR * NP; i += kThreads) {
                const int ti = i / NP, n = i % NP, t = run * TR + ti;
                if (t >= nt || n >= N) continue;
                float sqv = 0.f, skv = 0.f;
#pragma unroll
                for (int wv = 0; wv < kWarps; ++wv) {
                    sqv += rq[(ti * kWarps + wv) * NP + n];
                    skv += rk[(ti * kWarps + wv) * NP + n];
                }
                const int64_t at = (((int64_t)slice * ntok + tok0 + t0 + t) * H + h) * N + n;
                if (!SSM_BOUNDS(at, p.slices * ntok * H * N, BS_DELTA_SHARE)) continue;
                p.pq[at] = sqv;
                p.pk[at] = skv;
            }
            if (threadIdx.x < TR && run * TR + (int)threadIdx.x < nt) {
                const int ti = threadIdx.x;
                float sg = 0.f, sb = 0.f;
#pragma unroll
                for (int wv = 0; wv < kWarps; ++wv) {
                    sg += rg[ti * kWarps + wv];
                    sb += rb[ti * kWarps + wv];
                }
                const int64_t at = ((int64_t)slice * ntok + tok0 + t0 + run * TR + ti) * H + h;
                if (SSM_BOUNDS(at, p.slices * ntok * H, BS_DELTA_SHARE)) {
                    p.pg[at] = sg;
                    p.pb[at] = sb;
                }
            }
            __syncthreads();
        }
    }
    if (p.b.dh0 && live) {
        float *o = p.b.dh0 + srow * N;
#pragma unroll
        for (int e = 0; e < NE; ++e)
            if (state_of<L>(lrow, e) < N) o[state_of<L>(lrow, e)] = d[e];
    }
}

// Sum over the rows of a warp of 4 values per lane (one row, or two rows of 16
// lanes, which end with two values each), and where they go.
template <int L> constexpr int kRowKept = L == 32 ? 4 : 2;
template <int L> SSM_DEVINL void pair_sum(const float (&x)[4], float (&out)[kRowKept<L>], int lane) {
    static_assert(L == 32 || L == 16, "one or two rows a warp");
    if constexpr (L == 32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = x[e];
    } else {
        const bool hi = lane & 16;
#pragma unroll
        for (int e = 0; e < 2; ++e) out[e] = (hi ? x[e + 2] : x[e]) + __shfl_xor_sync(~0u, hi ? x[e] : x[e + 2], 16);
    }
}
template <int L> SSM_DEVINL void keep_pair(float *dst, const float (&v)[kRowKept<L>], int lane) {
    if constexpr (L == 32) *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<float2 *>(dst + (lane & 16 ? 2 : 0)) = make_float2(v[0], v[1]);
}

// The same for few rows and dstate <= 4 L: w = a h_{t-1} of all 32 tokens between
// two checkpoints fits in shared memory, so the states are walked once, in loops
// short enough for the instruction cache.  The next token's operands are read
// while a token's sum runs, the next tokens' rows while the tokens before are in
// work.  The shares of kGroup tokens at a time are added over the CTA's warps,
// out of two buffers in turn.
constexpr int kGroup = 8;
template <int L, int W> constexpr int rows_bwd_floats() {
    constexpr int NP = 4 * L, R = Cut<L, W>::rows, K = kDeltaCkpt;
    return 2 * K * NP + K * R * NP + 4 * K * R + 2 * K + 2 * kGroup * (2 * W * NP + W * 32 + R);
}

template <typename T, int L, int W>
__global__ void __launch_bounds__(W * 32, 1) delta_rows_bwd_kernel(const BwdArgs p) {
    constexpr int kThreads = W * 32, kRows = Cut<L, W>::rows, kTok = kDeltaCkpt, NE = 4, NP = NE * L;
    const ssm_delta_args &a = p.b.fwd;
    if (p.sv.err && *p.sv.err != 0) return;
    extern __shared__ float sm[];
    float *ks = sm, *qs = ks + kTok * NP, *ws = qs + kTok * NP;        // ws [kTok][kRows][NP]
    float *vs = ws + kTok * kRows * NP, *ds = vs + kTok * kRows, *us = ds + kTok * kRows, *es = us + kTok * kRows;
    float *as = es + kTok * kRows, *bs = as + kTok;
    float *rq = bs + kTok, *rk = rq + 2 * kGroup * W * NP;             // [2][kGroup][W][NP]
    float *rg = rk + 2 * kGroup * W * NP, *rb = rg + 2 * kGroup * kThreads;    // [2][kGroup][threads], [2][kGroup][kRows]
    const Seq sq = find_seq(a, p.sv, blockIdx.y);
    const int64_t H = a.nheads, P = a.headdim, N = a.dstate;
    const int h = blockIdx.x % H, slice = (int)(blockIdx.x / H), p0 = slice * kRows;
    const int grp = (int)(h / (H / a.ngroups));
    if (!SSM_BOUNDS(sq.hi, a.seqlen + 1, BS_DELTA_SEQ) || !SSM_BOUNDS(sq.lo, sq.hi + 1, BS_DELTA_SEQ)) return;
    if (!SSM_BOUNDS(sq.ckpt_row + (sq.hi - sq.lo + kTok - 1) / kTok, p.ckpt_rows + 1, BS_DELTA_CKPT) ||
        !SSM_BOUNDS(p0, P, BS_DELTA_STATE) || !SSM_BOUNDS(slice, p.slices, BS_DELTA_SHARE)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lrow = lane % L;
    const int r = warp * Cut<L, W>::per_warp + lane / L, n0 = lrow * 4;    // this lane's row and first state
    const bool live = p0 + r < P;
    const int64_t srow = ((int64_t)sq.s * H + h) * P + p0 + r;
    float d[NE] = {0.f, 0.f, 0.f, 0.f};
    if (live && p.b.dh_final) load_row<NE, L>(d, p.b.dh_final + srow * N, lrow, N);
    const T *q = (const T *)a.q + sq.row * a.q_batch_stride + grp * N;
    const T *k = (const T *)a.k + sq.row * a.k_batch_stride + grp * N;
    const T *v = (const T *)a.v + sq.row * a.v_batch_stride + h * P + p0;
    const T *dy = (const T *)p.b.dy + sq.row * p.b.dy_batch_stride + h * P + p0;
    const float *g = a.g + sq.row * a.g_batch_stride + h, *be = a.beta + sq.row * a.beta_batch_stride + h;
    const int64_t tok0 = sq.row * a.seqlen, ntok = a.batch * a.seqlen;
    T *dv = (T *)p.b.dv + h * P + p0;
    const int vw = (int)min((int64_t)kRows, P - p0);
    const int64_t len = sq.hi - sq.lo, chunks = (len + kTok - 1) / kTok;

    Staged<T, NP, kTok, kThreads> sk, sq_;
    Staged<T, kRows, kTok, kThreads> sv, sd;
    float ga = 1.f, gb = 0.f, st0[NE];
    const auto fetch = [&](int64_t c) {
        const int64_t t0 = sq.lo + c * kTok;
        const int nt = (int)min((int64_t)kTok, sq.hi - t0);
        sk.load(k + t0 * a.k_token_stride, a.k_token_stride, nt, (int)N);
        sq_.load(q + t0 * a.q_token_stride, a.q_token_stride, nt, (int)N);
        sv.load(v + t0 * a.v_token_stride, a.v_token_stride, nt, vw);
        sd.load(dy + t0 * p.b.dy_token_stride, p.b.dy_token_stride, nt, vw);
        if (threadIdx.x < kTok) {
            const int t = threadIdx.x;
            ga = t < nt ? g[(t0 + t) * a.g_token_stride] : 0.f;
            gb = t < nt ? be[(t0 + t) * a.beta_token_stride] : 0.f;
        }
        if (live) load_row<NE, L>(st0, p.ckpt + (((sq.ckpt_row + c) * H + h) * P + p0 + r) * N, lrow, N);
        else
#pragma unroll
            for (int e = 0; e < NE; ++e) st0[e] = 0.f;
    };
    const auto at4 = [&](const float *x) { return *reinterpret_cast<const float4 *>(x + n0); };
    if (chunks > 0) fetch(chunks - 1);
    for (int64_t c = chunks - 1; c >= 0; --c) {
        const int64_t t0 = sq.lo + c * kTok;
        const int nt = (int)min((int64_t)kTok, sq.hi - t0);
        __syncthreads();                               // the tokens before are done with
        sk.store(ks);
        sq_.store(qs);
        sv.store(vs);
        sd.store(ds);
        if (threadIdx.x < kTok) {
            as[threadIdx.x] = decay_of(ga);
            bs[threadIdx.x] = gb;
        }
        float st[NE];
#pragma unroll
        for (int e = 0; e < NE; ++e) st[e] = st0[e];
        __syncthreads();
        if (c > 0) fetch(c - 1);
        {   // w, u and v - w k of every token
            float4 kn = at4(ks);
            float an = as[0], bn = bs[0], vn = vs[r];
#pragma unroll 2
            for (int t = 0; t < nt; ++t) {
                const float4 k4 = kn;
                const float bt = bn, vt = vn;
                const float4 w = make_float4(st[0] * an, st[1] * an, st[2] * an, st[3] * an);
                const int tn = min(t + 1, kTok - 1);
                kn = at4(ks + tn * NP);
                an = as[tn];
                bn = bs[tn];
                vn = vs[tn * kRows + r];
                *reinterpret_cast<float4 *>(ws + (t * kRows + r) * NP + n0) = w;
                const float e = vt - row_sum<L>(fmaf(w.x, k4.x, w.y * k4.y) + fmaf(w.z, k4.z, w.w * k4.w));
                const float u = bt * e;
                st[0] = fmaf(u, k4.x, w.x);
                st[1] = fmaf(u, k4.y, w.y);
                st[2] = fmaf(u, k4.z, w.z);
                st[3] = fmaf(u, k4.w, w.w);
                if (lrow == 0) {
                    us[t * kRows + r] = u;
                    es[t * kRows + r] = e;
                }
            }
        }
        __syncwarp();                                  // (rows, and with them us and es, belong to one warp)
        float4 kn, qn, wn;
        float an, bn, un, en, yn;
        const auto token = [&](int t) {
            kn = at4(ks + t * NP);
            qn = at4(qs + t * NP);
            wn = at4(ws + (t * kRows + r) * NP);
            an = as[t];
            bn = bs[t];
            un = us[t * kRows + r];
            en = es[t * kRows + r];
            yn = a.scale * ds[t * kRows + r];
        };
        token(nt - 1);
        for (int grp8 = (nt - 1) / kGroup; grp8 >= 0; --grp8) {
            const int buf = grp8 & 1, first = grp8 * kGroup, cnt = min(kGroup, nt - first);
            float *bq = rq + buf * kGroup * W * NP, *bk = rk + buf * kGroup * W * NP, *bg = rg + buf * kGroup * kThreads,
                  *bb = rb + buf * kGroup * kRows;
#pragma unroll 2
            for (int i = cnt - 1; i >= 0; --i) {
                const int t = first + i;
                const float kk[NE] = {kn.x, kn.y, kn.z, kn.w}, qq[NE] = {qn.x, qn.y, qn.z, qn.w},
                            w[NE] = {wn.x, wn.y, wn.z, wn.w};
                const float al = an, bt = bn, u = un, ev = en, dyv = yn;
                token(max(t - 1, 0));
                float x[NE], part[kRowKept<L>];
#pragma unroll
                for (int e = 0; e < NE; ++e) d[e] = fmaf(dyv, qq[e], d[e]);
                const float du = row_sum<L>(fmaf(d[0], kk[0], d[1] * kk[1]) + fmaf(d[2], kk[2], d[3] * kk[3]));
                const int slot = (i * W + warp) * NP + n0;
#pragma unroll
                for (int e = 0; e < NE; ++e) x[e] = dyv * fmaf(u, kk[e], w[e]);        // dq: dy h_t
                pair_sum<L>(x, part, lane);
                keep_pair<L>(bq + slot, part, lane);
                const float dsv = -bt * du;
                float dg = 0.f;
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    x[e] = fmaf(u, d[e], dsv * w[e]);
                    d[e] = fmaf(dsv, kk[e], d[e]);
                    dg = fmaf(d[e], w[e], dg);
                    d[e] *= al;
                }
                pair_sum<L>(x, part, lane);
                keep_pair<L>(bk + slot, part, lane);
                bg[i * kThreads + threadIdx.x] = dg;
                if (lrow == 0) {
                    bb[i * kRows + r] = du * ev;
                    if (live) Elem<T>::st(dv + (tok0 + t0 + t) * H * P + r, -dsv);
                }
            }
            __syncthreads();                           // (the other buffer's readers are past the one before)
            for (int i = threadIdx.x; i < cnt * NP; i += kThreads) {
                const int ti = i / NP, n = i % NP;
                if (n >= N) continue;
                float sqv = 0.f, skv = 0.f;
#pragma unroll
                for (int wv = 0; wv < W; ++wv) {
                    sqv += bq[(ti * W + wv) * NP + n];
                    skv += bk[(ti * W + wv) * NP + n];
                }
                const int64_t at = (((int64_t)slice * ntok + tok0 + t0 + first + ti) * H + h) * N + n;
                if (!SSM_BOUNDS(at, p.slices * ntok * H * N, BS_DELTA_SHARE)) continue;
                p.pq[at] = sqv;
                p.pk[at] = skv;
            }
            for (int ti = warp; ti < cnt; ti += W) {
                float sg = 0.f, sb = lane < kRows ? bb[ti * kRows + lane] : 0.f;
#pragma unroll
                for (int i = 0; i < W; ++i) sg += bg[ti * kThreads + i * 32 + lane];
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    sg += __shfl_xor_sync(~0u, sg, o);
                    sb += __shfl_xor_sync(~0u, sb, o);
                }
                if (lane == 0) {
                    const int64_t at = ((int64_t)slice * ntok + tok0 + t0 + first + ti) * H + h;
                    if (SSM_BOUNDS(at, p.slices * ntok * H, BS_DELTA_SHARE)) {
                        p.pg[at] = sg;
                        p.pb[at] = sb;
                    }
                }
            }
        }
    }
    if (live && p.b.dh0)
#pragma unroll
        for (int e = 0; e < NE; ++e)
            if (n0 + e < N) p.b.dh0[srow * N + n0 + e] = d[e];
}

// Adds the shares of the row slices and, for dq / dk, of a group's heads.
template <typename T>
__global__ void delta_shares_kernel(const BwdArgs p, int slices) {
    if (p.sv.err && *p.sv.err != 0) return;
    const ssm_delta_args &a = p.b.fwd;
    const int64_t H = a.nheads, N = a.dstate, G = a.ngroups, R = H / G, ntok = a.batch * a.seqlen;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x, first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    for (int64_t i = first; i < ntok * G * N; i += stride) {
        const int64_t n = i % N, gt = i / N, grp = gt % G, t = gt / G;
        float sq = 0.f, sk = 0.f;
        for (int s = 0; s < slices; ++s)
            for (int64_t j = 0; j < R; ++j) {
                const int64_t at = (((int64_t)s * ntok + t) * H + grp * R + j) * N + n;
                sq += p.pq[at];
                sk += p.pk[at];
            }
        Elem<T>::st((T *)p.b.dq + i, sq);
        Elem<T>::st((T *)p.b.dk + i, sk);
    }
    for (int64_t i = first; i < ntok * H; i += stride) {
        float sg = 0.f, sb = 0.f;
        for (int s = 0; s < slices; ++s) {
            sg += p.pg[(int64_t)s * ntok * H + i];
            sb += p.pb[(int64_t)s * ntok * H + i];
        }
        store_gates<T>(p.b, i, sg, sb);
    }
}

template <typename K>
cudaError_t set_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int NE, int L, int W, bool Y>
cudaError_t run_scan(const Args &p, cudaStream_t st) {
    constexpr int kRows = Cut<L, W>::rows;
    const ssm_delta_args &a = p.a;
    const dim3 grid((unsigned)(a.nheads * ((a.headdim + kRows - 1) / kRows)), (unsigned)(a.cu_seqlens ? a.nseqs : a.batch));
    const size_t smem = (size_t)scan_floats<NE, L, W, Y>() * 4;
    cudaError_t e = set_smem(delta_scan_kernel<T, NE, L, W, Y>, smem);
    if (e != cudaSuccess) return e;
    delta_scan_kernel<T, NE, L, W, Y><<<grid, W * 32, smem, st>>>(p);
    return cudaGetLastError();
}
template <typename T, int NE, int L, int W>
cudaError_t run_fwd(const Args &p, cudaStream_t st) {
    return p.a.y ? run_scan<T, NE, L, W, true>(p, st) : run_scan<T, NE, L, W, false>(p, st);
}
template <typename T, int NE, int TR, int L, int W>
cudaError_t run_bwd(const BwdArgs &p, cudaStream_t st) {
    constexpr int kTok = kDeltaCkpt, kRows = Cut<L, W>::rows;
    const ssm_delta_args &a = p.b.fwd;
    const dim3 grid((unsigned)(a.nheads * ((a.headdim + kRows - 1) / kRows)), (unsigned)(a.cu_seqlens ? a.nseqs : a.batch));
    const size_t smem = (size_t)(2 * kTok * NE * L + 2 * kTok * kRows + 2 * kTok + 2 * TR * W * NE * L + 2 * TR * W) * 4;
    cudaError_t e = set_smem(delta_scan_bwd_kernel<T, NE, TR, L, W>, smem);
    if (e != cudaSuccess) return e;
    delta_scan_bwd_kernel<T, NE, TR, L, W><<<grid, W * 32, smem, st>>>(p);
    return cudaGetLastError();
}

template <typename T, int L, int W>
cudaError_t run_rows_bwd(const BwdArgs &p, cudaStream_t st) {
    constexpr int kRows = Cut<L, W>::rows;
    const ssm_delta_args &a = p.b.fwd;
    const dim3 grid((unsigned)(a.nheads * ((a.headdim + kRows - 1) / kRows)), (unsigned)(a.cu_seqlens ? a.nseqs : a.batch));
    constexpr size_t smem = (size_t)rows_bwd_floats<L, W>() * 4;
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    cudaError_t e = set_smem(delta_rows_bwd_kernel<T, L, W>, smem);
    if (e != cudaSuccess) return e;
    delta_rows_bwd_kernel<T, L, W><<<grid, W * 32, smem, st>>>(p);
    return cudaGetLastError();
}

int64_t seqs_of(const ssm_delta_args &a) { return a.cu_seqlens ? a.nseqs : a.batch; }
// Few rows: CTAs of 4 warps with a row in 16 (dstate <= 64) or 32 lanes fit on the
// SMs at once.  The chain is latency there, and a quarter of the states per lane
// shortens a token; with more rows the shuffles and copies of k and q cost more
// than that gains.  Forward / backward in us, few-row form against the other:
// 2 x 333 tokens, 6 heads, P 40, N 72 (480 rows) 62 / 245 against 82 / 400;
// 2 x 512, 16 heads, P 64, N 64 (2048 rows) 96 / 556 against 96 / 470;
// 4 x 256, 16 heads, P 64, N 64 (4096 rows) 68 / 536 against 53 / 247.
int64_t few_slices(const ssm_delta_args &a) {
    const int rows = a.dstate <= 64 ? Cut<16, 4>::rows : Cut<32, 4>::rows;
    return (a.headdim + rows - 1) / rows;
}
bool few_rows(const ssm_delta_args &a) { return seqs_of(a) * a.nheads * few_slices(a) <= sm_count(); }
int64_t slices_of(const ssm_delta_args &a) {
    return few_rows(a) ? few_slices(a) : (a.headdim + Cut<8, 8>::rows - 1) / Cut<8, 8>::rows;
}
template <typename T>
cudaError_t pick_fwd(const Args &p, cudaStream_t st) {
    const int64_t N = p.a.dstate;
    if (few_rows(p.a) && N <= 64) return run_fwd<T, 4, 16, 4>(p, st);
    if (few_rows(p.a)) return N <= 128 ? run_fwd<T, 8, 16, 4>(p, st) : run_fwd<T, 8, 32, 4>(p, st);
    if (N <= 32) return run_fwd<T, 4, 8, 8>(p, st);
    if (N <= 64) return run_fwd<T, 8, 8, 8>(p, st);
    if (N <= 96) return run_fwd<T, 12, 8, 8>(p, st);
    return N <= 128 ? run_fwd<T, 16, 8, 8>(p, st) : run_fwd<T, 32, 8, 8>(p, st);
}
template <typename T>
cudaError_t pick_bwd(const BwdArgs &p, cudaStream_t st) {
    const int64_t N = p.b.fwd.dstate;
    if (few_rows(p.b.fwd) && N <= 64) return run_rows_bwd<T, 16, 4>(p, st);
    if (few_rows(p.b.fwd)) return N <= 128 ? run_rows_bwd<T, 32, 4>(p, st) : run_bwd<T, 8, 8, 32, 4>(p, st);
    if (N <= 32) return run_bwd<T, 4, 8, 8, 8>(p, st);
    if (N <= 64) return run_bwd<T, 8, 8, 8, 8>(p, st);
    if (N <= 96) return run_bwd<T, 12, 8, 8, 8>(p, st);
    return N <= 128 ? run_bwd<T, 16, 8, 8, 8>(p, st) : run_bwd<T, 32, 4, 8, 8>(p, st);
}
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_delta_simt(const ssm_delta_args &a, const SeqView &sv, float *ckpt, cudaStream_t st) {
    if (seqs_of(a) == 0) return cudaSuccess;
    const Args p{a, sv, ckpt, delta_ckpt_rows(a)};
    return a.dtype == SSM_BF16 ? pick_fwd<__nv_bfloat16>(p, st) : pick_fwd<float>(p, st);
}

size_t delta_simt_bwd_workspace_bytes(const ssm_delta_bwd_args &b) {
    const ssm_delta_args &a = b.fwd;
    const size_t tok = (size_t)(a.batch * a.seqlen) * a.nheads * slices_of(a) * 4;
    return up256((size_t)delta_ckpt_rows(a) * a.nheads * a.headdim * a.dstate * 4) + 2 * up256(tok * a.dstate) +
           2 * up256(tok);
}

cudaError_t launch_delta_simt_bwd(const ssm_delta_bwd_args &b, const SeqView &sv, void *ws, cudaStream_t st) {
    const ssm_delta_args &a = b.fwd;
    if (seqs_of(a) == 0) return cudaSuccess;
    char *at = static_cast<char *>(ws);
    float *ckpt = reinterpret_cast<float *>(at);
    at += up256((size_t)delta_ckpt_rows(a) * a.nheads * a.headdim * a.dstate * 4);
    const size_t tok = (size_t)(a.batch * a.seqlen) * a.nheads * slices_of(a) * 4;
    BwdArgs p{b, sv, ckpt, nullptr, nullptr, nullptr, nullptr, delta_ckpt_rows(a), slices_of(a)};
    p.pq = reinterpret_cast<float *>(at); at += up256(tok * a.dstate);
    p.pk = reinterpret_cast<float *>(at); at += up256(tok * a.dstate);
    p.pg = reinterpret_cast<float *>(at); at += up256(tok);
    p.pb = reinterpret_cast<float *>(at);
    ssm_delta_args f = a;
    f.y = nullptr;
    f.h_final = nullptr;
    cudaError_t e = launch_delta_simt(f, sv, ckpt, st);
    if (e != cudaSuccess) return e;
    const bool bf = a.dtype == SSM_BF16;
    e = bf ? pick_bwd<__nv_bfloat16>(p, st) : pick_bwd<float>(p, st);
    if (e != cudaSuccess) return e;
    const int64_t work = a.batch * a.seqlen * a.ngroups * a.dstate;
    if (work == 0) return cudaSuccess;
    const int blocks = (int)min((work + 255) / 256, (int64_t)sm_count() * 8);
    if (bf) delta_shares_kernel<__nv_bfloat16><<<blocks, 256, 0, st>>>(p, (int)slices_of(a));
    else delta_shares_kernel<float><<<blocks, 256, 0, st>>>(p, (int)slices_of(a));
    return cudaGetLastError();
}

}  // namespace ssm
