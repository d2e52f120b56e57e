// state_pages.cu -- pages of a recurrent-state cache: copy, fork, free and
// compact (semantics in ssm.h).
//
// Two launches: one CTA plans (which pages go where, all rules about invalid
// and conflicting entries, reference counts and tables), then as many CTAs as
// fill the GPU move 16 KiB pieces of the planned pages (HBM-bound: each byte
// is read once and written once).  The plan only leaves moves whose
// destinations no move reads and no other move writes, so the pieces may go
// in any order.  96 pages of 2.1 MB forked from 256 live ones: 68 us for the
// move (384 MB, 5.6 TB/s) behind 3 us of planning.
#include "common.cuh"
#include "pages.h"

namespace ssm {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int64_t kPiece = 16384;

// Workspace: [0, 256) error word and move count; then mark, from, to (int32).
struct Ws {
    int32_t *err, *count, *mark, *from, *to;
};
Ws ws_of(const ssm_pages_args &a, void *ws) {
    char *w = static_cast<char *>(ws);
    const int64_t m = a.n > a.nslots ? a.n : a.nslots;
    Ws r;
    r.err = reinterpret_cast<int32_t *>(w);
    r.count = r.err + 1;
    r.mark = reinterpret_cast<int32_t *>(w + 256);
    r.from = r.mark + 2 * a.nslots;
    r.to = r.from + m;
    return r;
}

// Exclusive prefix sum of one value per thread over the CTA; `total` gets the sum.
SSM_DEVINL int scan_cta(int v, int *sm, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sm[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int y = sm[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(~0u, y, o);
            if (lane >= o) y += z;
        }
        sm[lane] = y;
    }
    __syncthreads();
    total = sm[31];
    return x - v + (warp ? sm[warp - 1] : 0);
}

// Calls f(i, rank) for every i < n with pred(i), rank counting them in order.
// Blocks of kPlanThreads indices at a time, so that reads are coalesced.
template <typename Pred, typename F>
SSM_DEVINL int ranked(int64_t n, int *sm, Pred pred, F f) {
    int base = 0;
    for (int64_t i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int64_t i = i0 + threadIdx.x;
        const bool in = i < n && pred(i);
        int total;
        const int rank = base + scan_cta(in, sm, total);
        if (in) f(i, rank);
        base += total;
    }
    return base;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PageOp op, const ssm_pages_args a, const Ws w) {
    __shared__ int sm[32];
    const int32_t ns = (int32_t)a.nslots;
    const int tid = threadIdx.x;
    int bad = 0;
    if (op == PageOp::kCopy) {
        // mark[p]: the first entry that writes page p; mark[ns + p]: an entry reads it
        for (int p = tid; p < ns; p += kPlanThreads) {
            w.mark[p] = INT32_MAX;
            w.mark[ns + p] = 0;
        }
        __syncthreads();
        for (int64_t i = tid; i < a.n; i += kPlanThreads) {
            const int s = a.src[i], d = a.pages[i];
            if (d < 0 || s == d) continue;
            if (s < -1 || s >= ns || d >= ns) { bad = 1; continue; }
            atomicMin(w.mark + d, (int)i);
            if (s >= 0) atomicOr(w.mark + ns + s, 1);
        }
        __syncthreads();
        for (int64_t i = tid; i < a.n; i += kPlanThreads) {
            const int s = a.src[i], d = a.pages[i];
            bool ok = d >= 0 && s != d && s >= -1 && s < ns && d < ns;
            if (ok && (w.mark[d] != (int)i || w.mark[ns + d])) { ok = false; bad = 1; }
            w.from[i] = s;
            w.to[i] = ok ? d : -1;
        }
        if (tid == 0) *w.count = (int)a.n;
    } else if (op == PageOp::kFork) {
        // the free pages in order, then one for every valid entry in order
        const int nfree = ranked(ns, sm, [&](int64_t p) { return a.refs[p] == 0; },
                                 [&](int64_t p, int rank) { w.mark[rank] = (int)p; });
        __syncthreads();
        const auto valid = [&](int64_t i) {
            const int s = w.from[i];
            return s == -1 || (s >= 0 && s < ns && a.refs[s] > 0);
        };
        for (int64_t i = tid; i < a.n; i += kPlanThreads) {
            w.from[i] = a.src[i];                      // (pages may be src)
            a.pages[i] = -1;
            w.to[i] = -1;
            if (!valid(i)) bad = 1;
        }
        __syncthreads();
        ranked(a.n, sm, valid, [&](int64_t i, int rank) {
            if (rank < nfree) w.to[i] = w.mark[rank];
            else bad = 1;
        });
        __syncthreads();               // every entry has read refs
        for (int64_t i = tid; i < a.n; i += kPlanThreads)
            if (w.to[i] >= 0) {
                a.pages[i] = w.to[i];
                a.refs[w.to[i]] = 1;
            }
        if (tid == 0) *w.count = (int)a.n;
    } else if (op == PageOp::kFree) {
        for (int64_t i = tid; i < a.n; i += kPlanThreads) {
            const int p = a.pages[i];
            if (p < 0) continue;
            if (p >= ns) { bad = 1; continue; }
            if (atomicSub(a.refs + p, 1) <= 0) {       // not held: put back what was taken
                atomicAdd(a.refs + p, 1);
                bad = 1;
            }
        }
    } else {
        const auto live = [&](int64_t p) { return a.refs[p] > 0; };
        const int n = ranked(ns, sm, live, [&](int64_t, int) {});
        // mark[p]: the new number of live page p (-1: not live); to / from: the moves
        ranked(n, sm, [&](int64_t p) { return !live(p); }, [&](int64_t p, int rank) { w.to[rank] = (int)p; });
        __syncthreads();
        for (int p = tid; p < ns; p += kPlanThreads) w.mark[p] = live(p) ? p : -1;
        __syncthreads();
        const int moves = ranked(ns - n, sm, [&](int64_t i) { return live(n + i); },
                                 [&](int64_t i, int rank) {
                                     w.from[rank] = (int)(n + i);
                                     w.mark[n + i] = w.to[rank];
                                 });
        __syncthreads();
        for (int i = tid; i < moves; i += kPlanThreads) {
            a.refs[w.to[i]] = a.refs[w.from[i]];
            a.refs[w.from[i]] = 0;
        }
        for (int64_t j = tid; j < a.n; j += kPlanThreads) {
            const int p = a.pages[j];
            if (p < 0) continue;
            const int q = p < ns ? w.mark[p] : -1;
            if (q < 0) bad = 1;
            if (q != p) a.pages[j] = q;
        }
        if (tid == 0) *w.count = moves;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) *w.err = bad ? SSM_DEVERR_PAGES : SSM_DEVERR_NONE;
}

template <typename V>
SSM_DEVINL void move_piece(const char *src, char *dst, int64_t bytes, bool zero) {
    constexpr int U = 4;                       // loads in flight per thread
    const int64_t n = bytes / (int64_t)sizeof(V);
    const V *s = reinterpret_cast<const V *>(src);
    V *d = reinterpret_cast<V *>(dst);
    for (int64_t i = threadIdx.x; i < n; i += (int64_t)U * kMoveThreads) {
        V v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * kMoveThreads < n) v[u] = zero ? V{} : s[i + u * kMoveThreads];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * kMoveThreads < n) d[i + u * kMoveThreads] = v[u];
    }
}

struct Pieces {
    int64_t first[SSM_MAX_POOLS + 1];          // pieces of the pools before, of one page
};

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const ssm_pages_args a, const Ws w, const Pieces pc) {
    const int64_t per = pc.first[a.npools], total = (int64_t)*w.count * per;
    for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
        const int64_t m = i / per, piece = i % per;
        const int to = w.to[m], from = w.from[m];
        if (to < 0) continue;
        if (!SSM_BOUNDS(to, a.nslots, BS_PAGE) || !SSM_BOUNDS(from + 1, a.nslots + 1, BS_PAGE)) continue;
        int k = 0;
        while (piece >= pc.first[k + 1]) ++k;
        const int64_t pb = a.pools[k].page_bytes, off = (piece - pc.first[k]) * kPiece;
        const int64_t bytes = min(kPiece, pb - off);
        char *base = static_cast<char *>(a.pools[k].base);
        char *dst = base + (int64_t)to * pb + off;
        const char *src = base + (int64_t)(from < 0 ? 0 : from) * pb + off;
        const uint64_t al = (uint64_t)base | (uint64_t)pb;
        if (al % 16 == 0) move_piece<uint4>(src, dst, bytes, from < 0);
        else if (al % 4 == 0) move_piece<uint32_t>(src, dst, bytes, from < 0);
        else if (al % 2 == 0) move_piece<uint16_t>(src, dst, bytes, from < 0);
        else move_piece<uint8_t>(src, dst, bytes, from < 0);
    }
}

}  // namespace

size_t pages_workspace_bytes(const ssm_pages_args &a) {
    const int64_t m = a.n > a.nslots ? a.n : a.nslots;
    return 256 + ((size_t)(2 * a.nslots + 2 * m) * 4 + 255) / 256 * 256;
}

cudaError_t launch_pages(PageOp op, const ssm_pages_args &a, void *ws, cudaStream_t st) {
    const Ws w = ws_of(a, ws);
    plan_kernel<<<1, kPlanThreads, 0, st>>>(op, a, w);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || op == PageOp::kFree || a.npools == 0) return e;
    Pieces pc;
    pc.first[0] = 0;
    for (int k = 0; k < a.npools; ++k) pc.first[k + 1] = pc.first[k] + (a.pools[k].page_bytes + kPiece - 1) / kPiece;
    // compaction moves at most half the slots
    const int64_t most = (op == PageOp::kCompact ? a.nslots / 2 : a.n) * pc.first[a.npools];
    if (most == 0) return cudaSuccess;
    const int64_t grid = (int64_t)sm_count() * 8;
    timing_begin(st);
    move_kernel<<<(unsigned)(most < grid ? most : grid), kMoveThreads, 0, st>>>(a, w, pc);
    timing_end(st);
    return cudaGetLastError();
}

}  // namespace ssm
