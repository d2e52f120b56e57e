// delta_tc.cuh -- pieces shared by the tensor-core kernels of the gated delta
// rule: block geometry, bounded waits, tensor-memory helpers, gate tables.
#pragma once

#include "common.cuh"
#include "delta.h"
#include "tc05.cuh"

namespace ssm {
namespace dtc {

constexpr int kQ = 64;                    // tokens per block
constexpr uint32_t kTile = 8192;          // 64 rows x 64 bf16: one 128-byte-swizzled tile
constexpr size_t kTBytes = 2 * kTile;     // T of one (block, head): high and low parts
// What the pre-pass leaves of one (block, head): T high, T low, attention weights
// (high); for the backward also their low part.
constexpr size_t kHeadBytes = 3 * kTile, kHeadBytesBwd = 4 * kTile;

// What the backward keeps of one (block, head, 64-row slice): the entering state
// and the gradient of the leaving state (64 rows x dstate, high parts), then
// dy, dR and u transposed (64 rows x 64 tokens).  Rows past headdim and tokens
// past the sequence are zero.  16 bytes of a row (8 columns) lie beside those
// of the next row: a warp, a row in each lane, writes whole lines (in rows of
// 128 bytes the same stores took a line each and were the chain's bound), and
// the tile is an unswizzled MN-major operand as it stands: 8 columns every
// 1024 bytes, 8 rows every 128.
SSM_DEVINL uint32_t rec_off(int row, int col) { return (uint32_t)(col >> 3) * 1024u + (uint32_t)row * 16u; }
struct Rec {
    uint8_t *base;
    int64_t state;                 // bytes of one state tile: 128 x dstate rounded up to 64
    int nsl;
    SSM_DEVINL uint8_t *at(int64_t slot, int64_t H, int head, int slice) const {
        return base + ((slot * H + head) * nsl + slice) * (2 * state + 3 * (int64_t)kTile);
    }
    SSM_DEVINL int64_t dy() const { return 2 * state; }
    SSM_DEVINL int64_t dR() const { return 2 * state + kTile; }
    SSM_DEVINL int64_t u() const { return 2 * state + 2 * (int64_t)kTile; }
};
// beta of the backward: dbeta_i = dR_i . u_i / beta_i, and u_i / beta_i stays
// exact for a beta so small that nothing else notices it.
constexpr float kTinyBeta = 1e-20f;
SSM_DEVINL float bwd_beta(float b) { return fabsf(b) < kTinyBeta ? copysignf(kTinyBeta, b) : b; }

// The first 1024-byte boundary of the dynamic shared memory, by an offset: a
// pointer made from an integer would turn every access into a generic one.
SSM_DEVINL uint8_t *smem_1024(uint8_t *raw) { return raw + ((0u - tc::smem_u32(raw)) & 1023u); }

// How long a wait lasts before it gives up, and one look at the barrier.  In the
// checked build the limit is a variable, so that a test can make waits run out
// (ssm_delta_wait_limit), and a look does not sleep, so that short limits hold.
#ifdef SSM_CHECK_BOUNDS
SSM_DEVINL uint64_t wait_limit_ns() { return *(volatile unsigned long long *)&g_delta_wait_ns; }
SSM_DEVINL bool poll(uint64_t *mb, uint32_t parity) { return tc::mbar_test_wait(mb, parity); }
#else
SSM_DEVINL uint64_t wait_limit_ns() { return 2000000000ull; }
SSM_DEVINL bool poll(uint64_t *mb, uint32_t parity) { return tc::mbar_try_wait(mb, parity); }
#endif
// Wait for an mbarrier phase, at most two seconds; gives up as soon as another
// thread of the CTA has (`abort`), and records the timeout in the error word.
// The loop is kept out of line: a kernel of many roles waits in dozens of
// places, and its loops have to stay within the instruction cache.
static __device__ __noinline__ bool wait_slow(uint64_t *mb, volatile int *abort, uint32_t parity, int32_t *err) {
    const uint64_t t0 = tc::globaltimer_ns();
    for (;;) {
        if (*abort) return false;
        if (poll(mb, parity)) return true;
        if (tc::globaltimer_ns() - t0 >= wait_limit_ns()) break;
    }
    *abort = 1;
    if (err) atomicExch(err, SSM_DEVERR_TIMEOUT);
    return false;
}
SSM_DEVINL bool wait_bar(uint64_t *mb, volatile int *abort, uint32_t parity, int32_t *err) {
    return poll(mb, parity) || wait_slow(mb, abort, parity, err);
}
// The same by a whole warp, whose lanes go on or give up together: what follows
// are instructions that a warp issues as one.
SSM_DEVINL bool wait_warp(uint64_t *mb, volatile int *abort, uint32_t parity, int32_t *err) {
    return __all_sync(~0u, wait_bar(mb, abort, parity, err));
}
// Barrier 1 over `threads` threads that also tells whether `ok` holds in all of
// them: warps that meet at a barrier give up together.
template <int threads>
SSM_DEVINL bool bar_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.and.pred q, 1, %2, p;\nselp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)ok), "n"(threads)
        : "memory");
    return r != 0;
}
SSM_DEVINL void arrive(uint64_t *mbar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(tc::smem_u32(mbar)) : "memory");
}

// A operand in tensor memory (row = lane, two bf16 of K per column); `skip`:
// lanes of the accumulator to leave alone, 32 per word.
SSM_DEVINL void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
SSM_DEVINL void mma_ts_lanes(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t skip_lo,
                             uint32_t skip_hi) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %5, %6, %6}, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(skip_lo), "r"(skip_hi));
}

SSM_DEVINL void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
SSM_DEVINL void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// A load in two steps, so that other loads may stand between them; the values
// pass through the wait, which keeps their uses behind it.
SSM_DEVINL void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
SSM_DEVINL void tmem_ld32_wait(uint32_t (&r)[32], float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
    asm volatile(""
                 : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31]));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
SSM_DEVINL void tmem_st16f(uint32_t taddr, const float (&v)[16]) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
    tmem_st16(taddr, r);
}
SSM_DEVINL void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
SSM_DEVINL void tmem_st32(uint32_t taddr, const float (&v)[32]) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
    tmem_st16(taddr, r);
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[16 + i]);
    tmem_st16(taddr + 16, r);
}
SSM_DEVINL void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Two bf16 parts of a float: high = nearest bf16, low = nearest bf16 of the
// rest; together 16 bits of mantissa, relative error at most 2^-17.
SSM_DEVINL uint32_t pack2(float a, float b) {
    __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&p);
}
SSM_DEVINL void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack2(a, b);
    lo = pack2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}
// 16 floats as operand columns: 8 columns of high parts at hi, of low parts at lo.
SSM_DEVINL void st_split16(uint32_t hi, uint32_t lo, const float *v) {
    uint32_t h[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) split2(v[2 * i], v[2 * i + 1], h[i], l[i]);
    tmem_st8(hi, h);
    tmem_st8(lo, l);
}
SSM_DEVINL void split32(const float (&v)[32], uint32_t (&hi)[16], uint32_t (&lo)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) split2(v[2 * i], v[2 * i + 1], hi[i], lo[i]);
}

// cp.async.bulk of a contiguous range, global -> shared.
SSM_DEVINL void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *mbar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
            tc::smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(tc::smem_u32(mbar))
        : "memory");
}
SSM_DEVINL void tma_load_4d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, uint64_t *mbar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];\n" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(tc::smem_u32(mbar))
        : "memory");
}

// Byte offset of (row, col) in a 64-row tile of 64 bf16 columns, 128-byte swizzle.
SSM_DEVINL uint32_t swz(int row, int col) {
    return (uint32_t)row * 128u + ((uint32_t)((col >> 3) ^ (row & 7)) << 4) + (uint32_t)(col & 7) * 2u;
}

// Prefix sums of the log decays of one block, by one warp: lane l holds tokens
// l and l + 32.  In 64 bits, because the decays between tokens are differences
// of sums that may be far from zero; tokens behind the sequence's end count 0.
SSM_DEVINL void block_cs(float g0, float g1, double &c0, double &c1, double &last) {
    const int lane = threadIdx.x & 31;
    c0 = g0;
    c1 = g1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(~0u, c0, o), y = __shfl_up_sync(~0u, c1, o);
        if (lane >= o) {
            c0 += x;
            c1 += y;
        }
    }
    c1 += __shfl_sync(~0u, c0, 31);
    last = __shfl_sync(~0u, c1, 31);
}
SSM_DEVINL float exp_d(double x) { return ex2((float)(x * 1.4426950408889634)); }

// The sequence and block of a slot of per-block data (seq_slot is its inverse; nt = 0: none).
struct Block {
    int s;          // sequence
    int64_t row;    // batch row
    int64_t t0;     // first token (within the row)
    int nt;         // tokens, 0: empty slot
};
SSM_DEVINL int64_t seq_slot(const int32_t *cu, int s, int64_t nblk) {
    return cu ? (int64_t)cu[s] / kQ + s : (int64_t)s * nblk;
}
SSM_DEVINL Block find_block(const int32_t *cu, int nseqs, int64_t seqlen, int64_t nblk, int64_t slot) {
    Block b;
    int64_t lo, hi, c;
    if (cu) {
        int l = 0, h = nseqs - 1;
        while (l < h) {
            const int m = (l + h + 1) >> 1;
            if ((int64_t)cu[m] / kQ + m <= slot) l = m;
            else h = m - 1;
        }
        b.s = l;
        b.row = 0;
        lo = cu[l];
        hi = cu[l + 1];
        c = slot - ((int64_t)cu[l] / kQ + l);
    } else {
        b.s = (int)(slot / nblk);
        b.row = b.s;
        lo = 0;
        hi = seqlen;
        c = slot % nblk;
    }
    b.t0 = lo + c * kQ;
    b.nt = (int)max((int64_t)0, min((int64_t)kQ, hi - b.t0));
    return b;
}

}  // namespace dtc

// Slots of per-block data: sequence s starts at slot cu[s] / 64 + s (a bound
// that needs no prefix sum over rounded-up lengths), batch row r at r * blocks.
inline int64_t delta_blocks_per_row(const ssm_delta_args &a) { return (a.seqlen + dtc::kQ - 1) / dtc::kQ; }
inline int64_t delta_slots(const ssm_delta_args &a) {
    return a.cu_seqlens ? a.seqlen / dtc::kQ + a.nseqs + 1 : a.batch * delta_blocks_per_row(a);
}

}  // namespace ssm
