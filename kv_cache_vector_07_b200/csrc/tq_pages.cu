// Pages of a cache shared, taken, compacted and freed on the device, so that
// a serving loop's bookkeeping stays in stream order and can be captured into
// a graph.  The state is the caller's: a reference count per block (0 = free),
// the block table and the lengths.
//
// Every call is one planning kernel (a single block: the tables are small and
// its phases need one another's results) and, where bytes move, one kernel
// that moves them by the plan's list of jobs.  Free pages are dealt lowest
// number first, in the order of the requests, so the tables that come out
// depend on nothing but the tables that went in; the only atomics are integer
// sums and minima, whose order does not show.
#include <climits>

#include <cuda_runtime.h>

#include "tq_chain.cuh"
#include "tq_dev.cuh"

namespace tq {
namespace {

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;

// Workspace pieces (int32), behind the 256-byte header whose second word is
// the number of jobs.
struct PlanWs {
    uint32_t *status;
    int32_t *n_jobs;
    int32_t *mark;      // [n_rows] first request that names the row
    int32_t *need;      // [n_rows] pages a request needs, -1 = skipped
    int32_t *start;     // [n_rows] its first rank among the pages dealt
    int32_t *len;       // [n_rows] compact: a request's tokens before
    int64_t *slot0;     // [n_rows] reserve: its first entry of slot_mapping
    int32_t *ids;       // [num_blocks] free pages, lowest first
    int4 *jobs;         // [num_blocks] fork: {from, to}; compact: {request, page, to, old length}
    int32_t *old;       // [n_rows][max_blocks] compact: a request's pages before
    int32_t *fresh;     // [n_rows][max_blocks] compact: rank of a fresh page in its request, -1 = stays
};

struct PoolArgs {
    int32_t *refs, *table, *lens;
    int num_blocks, max_blocks, n_rows, P;
    PlanWs ws;
};

__host__ __device__ inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

size_t carve(uint8_t *ws, int64_t num_blocks, int n_rows, int max_blocks, PlanWs *p) {
    size_t off = kWsHeader;
    auto take = [&](size_t bytes) { uint8_t *at = ws + off; off += up256(bytes); return at; };
    p->status = reinterpret_cast<uint32_t *>(ws);
    p->n_jobs = reinterpret_cast<int32_t *>(ws) + 1;
    p->mark = reinterpret_cast<int32_t *>(take(4 * size_t(n_rows)));
    p->need = reinterpret_cast<int32_t *>(take(4 * size_t(n_rows)));
    p->start = reinterpret_cast<int32_t *>(take(4 * size_t(n_rows)));
    p->len = reinterpret_cast<int32_t *>(take(4 * size_t(n_rows)));
    p->slot0 = reinterpret_cast<int64_t *>(take(8 * size_t(n_rows)));
    p->ids = reinterpret_cast<int32_t *>(take(4 * size_t(num_blocks)));
    p->jobs = reinterpret_cast<int4 *>(take(16 * size_t(num_blocks)));
    p->old = reinterpret_cast<int32_t *>(take(4 * size_t(n_rows) * size_t(max_blocks)));
    p->fresh = reinterpret_cast<int32_t *>(take(4 * size_t(n_rows) * size_t(max_blocks)));
    return off;
}

// What a planning block keeps in shared memory: the requests' numbers where
// they fit, so that a phase does not wait for the last one's trip to memory.
constexpr int kSharedRequests = 1024, kSharedRows = 4096;
struct PlanShared {
    int64_t part[kPlanWarps];
    int32_t mark[kSharedRows];
    int32_t need[kSharedRequests], start[kSharedRequests], len[kSharedRequests];
    uint32_t bad;       // status bits of the call
    int jobs;
};

// Exclusive sum of v over the block's threads; *total receives the sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, PlanShared &sh, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sh.part[warp] = x;
    __syncthreads();
    int64_t w = sh.part[lane];                       // kPlanWarps = 32: every warp sums the warps' sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w += y;
    }
    const int64_t before = __shfl_sync(kFull, w, warp) - sh.part[warp];
    *total = __shfl_sync(kFull, w, 31);
    __syncthreads();
    return before + x - v;
}

// start[i] = the sum of max(need, 0) before i; returns the sum over all.
__device__ int64_t deal_ranks(const int32_t *need, int32_t *start, int n, PlanShared &sh) {
    int64_t carry = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        const int64_t v = i < n ? max(need[i], 0) : 0;
        int64_t total;
        const int64_t at = carry + block_scan(v, sh, &total);
        if (i < n) start[i] = int(min(at, int64_t(INT_MAX)));
        carry += total;
    }
    __syncthreads();
    return carry;
}

// The lowest `want` free pages into ids, ascending; returns how many there
// are.  A thread looks at 16 counts a round: 200,000 pages are 13 rounds.
__device__ int find_free(const int32_t *refs, int num_blocks, int64_t want, int32_t *ids, PlanShared &sh) {
    constexpr int PER = 16;
    const bool wide = reinterpret_cast<uintptr_t>(refs) % 16 == 0;
    int64_t found = 0;
    for (int64_t b0 = 0; b0 < num_blocks && found < want; b0 += kPlanThreads * PER) {
        const int64_t b = b0 + int64_t(threadIdx.x) * PER;
        uint32_t is_free = 0;
        if (wide && b + PER <= num_blocks) {
            const int4 *at = reinterpret_cast<const int4 *>(refs + b);
            int4 v[PER / 4];
#pragma unroll
            for (int i = 0; i < PER / 4; ++i) v[i] = at[i];
#pragma unroll
            for (int i = 0; i < PER / 4; ++i)
                is_free |= (uint32_t(v[i].x == 0) | uint32_t(v[i].y == 0) << 1 | uint32_t(v[i].z == 0) << 2 |
                            uint32_t(v[i].w == 0) << 3) << (4 * i);
        } else {
            for (int i = 0; i < PER; ++i)
                if (b + i < num_blocks && refs[b + i] == 0) is_free |= 1u << i;
        }
        int64_t total;
        int64_t at = found + block_scan(__popc(is_free), sh, &total);
        for (uint32_t f = is_free; f && at < want; f &= f - 1) ids[at++] = int(b) + __ffs(f) - 1;
        found += total;
    }
    __syncthreads();
    return int(min(found, want));
}

__device__ __forceinline__ bool live_page(const PoolArgs &a, int id) {
    return id >= 0 && id < a.num_blocks && a.refs[id] > 0;
}

// One reference less; a count that is not positive stays and is reported.
__device__ __forceinline__ void release(const PoolArgs &a, int id) {
    if (id < 0 || id >= a.num_blocks) {
        atomicOr(a.ws.status, TQ_DEV_BLOCK_RANGE);
    } else if (atomicSub(&a.refs[id], 1) <= 0) {
        atomicAdd(&a.refs[id], 1);
        atomicOr(a.ws.status, TQ_DEV_BLOCK_RANGE);
    }
}

// mark[r] = the first request naming row r.
__device__ void mark_rows(const PoolArgs &a, const int32_t *rows, int n, int32_t *mark) {
    for (int r = threadIdx.x; r < a.n_rows; r += kPlanThreads) mark[r] = INT_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        if (rows[i] >= 0 && rows[i] < a.n_rows) atomicMin(&mark[rows[i]], i);
    __syncthreads();
}

// Whether all pages of row r are in range and in use (a warp's question).
__device__ __forceinline__ bool row_lives(const PoolArgs &a, int r, int pages) {
    const int lane = threadIdx.x & 31;
    const int32_t *row = a.table + int64_t(r) * a.max_blocks;
    bool ok = true;
#pragma unroll 4
    for (int j = lane; j < pages; j += 32) ok &= live_page(a, row[j]);
    return __all_sync(kFull, ok);
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(PoolArgs a, const int32_t *src, const int32_t *dst,
                                                                 int n) {
    __shared__ PlanShared sh;
    let_next_in();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool few = n <= kSharedRequests;
    int32_t *need = few ? sh.need : a.ws.need, *start = few ? sh.start : a.ws.start, *lens = few ? sh.len : a.ws.old;
    int32_t *mark = a.n_rows <= kSharedRows ? sh.mark : a.ws.mark;
    if (threadIdx.x == 0) sh.bad = 0;
    mark_rows(a, dst, n, mark);
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int s = src[i], d = dst[i];
        const int len = s >= 0 && s < a.n_rows ? a.lens[s] : -1;
        const bool ok = d >= 0 && d < a.n_rows && mark[d] == i && a.lens[d] == 0 && len >= 0 &&
                        len <= a.max_blocks * int64_t(a.P);
        need[i] = ok ? len % a.P != 0 : -1;
        lens[i] = len;                               // read here: rows that a later phase fills are empty now
        if (!ok) atomicOr(&sh.bad, TQ_DEV_ROW);
    }
    __syncthreads();
    for (int i = warp; i < n; i += kPlanWarps) {
        if (need[i] < 0) continue;
        const bool ok = row_lives(a, src[i], int((int64_t(lens[i]) + a.P - 1) / a.P));
        __syncwarp();
        if (!ok && lane == 0) {
            need[i] = -1;
            atomicOr(&sh.bad, TQ_DEV_BLOCK_RANGE);
        }
    }
    __syncthreads();
    const int64_t want = deal_ranks(need, start, n, sh);
    const int found = find_free(a.refs, a.num_blocks, want, a.ws.ids, sh);
    for (int i = warp; i < n; i += kPlanWarps) {
        const int nd = need[i], at = start[i];
        if (nd < 0) continue;
        if (nd > 0 && at >= found) {
            if (lane == 0) atomicOr(&sh.bad, TQ_DEV_NO_PAGES);
            continue;
        }
        const int len = lens[i], full = len / a.P;
        const int32_t *from = a.table + int64_t(src[i]) * a.max_blocks;
        int32_t *to = a.table + int64_t(dst[i]) * a.max_blocks;
#pragma unroll 4
        for (int j = lane; j < full; j += 32) {
            const int id = from[j];
            to[j] = id;
            atomicAdd(&a.refs[id], 1);
        }
        if (lane == 0) {
            if (nd) {
                const int id = a.ws.ids[at];
                a.ws.jobs[at] = make_int4(from[full], id, 0, 0);
                to[full] = id;
                a.refs[id] = 1;
            }
            a.lens[dst[i]] = len;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        *a.ws.n_jobs = found;                        // one page a request: every page found is dealt
        if (sh.bad) atomicOr(a.ws.status, sh.bad);
    }
}

// The layers' cache addresses travel as a kernel argument (1 KB a launch).
constexpr int kLayersPerLaunch = 128;
struct Layers {
    uint8_t *at[kLayersPerLaunch];
};

// Job's page copied in layer blockIdx.y; blockIdx.z takes a slice of it.
__global__ void __launch_bounds__(256) copy_pages_kernel(const __grid_constant__ Layers layers, PlanWs ws,
                                                         int64_t block_bytes) {
    wait_for_last();
    if (int(blockIdx.x) >= *ws.n_jobs) return;
    const int4 job = ws.jobs[blockIdx.x];
    uint8_t *base = layers.at[blockIdx.y];
    const uint4 *from = reinterpret_cast<const uint4 *>(base + job.x * block_bytes);
    uint4 *to = reinterpret_cast<uint4 *>(base + job.y * block_bytes);
    const int64_t n = block_bytes / 16, step = int64_t(gridDim.z) * 256;
    for (int64_t i = int64_t(blockIdx.z) * 256 + threadIdx.x; i < n; i += step) to[i] = from[i];
}

// ---------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------
// A row's pages and slots; the lanes of a warp, or one thread, share the row.
__device__ __forceinline__ void reserve_row(const PoolArgs &a, int b, int64_t add, int need, int rank, int64_t at,
                                            int32_t *slots, int first, int step) {
    const int64_t len = a.lens[b];
    const int pages = int((len + a.P - 1) / a.P);
    int32_t *row = a.table + int64_t(b) * a.max_blocks;
    for (int j = first; j < need; j += step) {
        const int id = a.ws.ids[rank + j];
        row[pages + j] = id;
        a.refs[id] = 1;
    }
    if (step > 1) __syncwarp();
    for (int64_t t = first; t < add; t += step) {
        const int64_t pos = len + t;
        slots[at + t] = row[pos / a.P] * a.P + int(pos % a.P);
    }
    if (step > 1) __syncwarp();
    if (first == 0) a.lens[b] = int(len + add);
}

__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(PoolArgs a, const int32_t *new_tokens,
                                                                    int32_t *slots, int64_t n_slots) {
    __shared__ PlanShared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool few = a.n_rows <= kSharedRequests;
    int32_t *need = few ? sh.need : a.ws.need, *start = few ? sh.start : a.ws.start;
    if (threadIdx.x == 0) sh.bad = 0;
    __syncthreads();
    int64_t first = 0;                                   // entries of slot_mapping before this chunk of rows
    for (int b0 = 0; b0 < a.n_rows; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        const int64_t add = b < a.n_rows ? max(new_tokens[b], 0) : 0;
        int64_t total;
        const int64_t at = first + block_scan(add, sh, &total);
        first += total;
        if (b >= a.n_rows) continue;
        int nd = -1;
        if (add > 0) {
            const int64_t len = a.lens[b], pages = (len + a.P - 1) / a.P, then = (len + add + a.P - 1) / a.P;
            uint32_t bad = 0;
            if (len < 0 || at + add > n_slots) bad = TQ_DEV_ROW;
            else if (then > a.max_blocks) bad = TQ_DEV_NO_PAGES;
            else if (len % a.P != 0) {
                // the page that is filled on belongs to this row alone
                const int id = a.table[int64_t(b) * a.max_blocks + pages - 1];
                if (!live_page(a, id)) bad = TQ_DEV_BLOCK_RANGE;
                else if (a.refs[id] != 1) bad = TQ_DEV_PAGE_SHARED;
            }
            if (bad) atomicOr(&sh.bad, bad);
            else nd = int(then - pages);
        }
        need[b] = nd;
        a.ws.slot0[b] = at;
    }
    __syncthreads();
    const int64_t want = deal_ranks(need, start, a.n_rows, sh);
    const int found = find_free(a.refs, a.num_blocks, want, a.ws.ids, sh);
    // a thread serves a row of few tokens (a decode step's), a warp the others
    constexpr int kFew = 4;
    for (int pass = 0; pass < 2; ++pass) {
        const int b1 = pass ? warp : int(threadIdx.x), stride = pass ? kPlanWarps : kPlanThreads;
        for (int b = b1; b < a.n_rows; b += stride) {
            const int64_t add = max(new_tokens[b], 0);
            if (add == 0 || (add > kFew) != (pass == 1)) continue;
            const int64_t at = a.ws.slot0[b];
            const int me = pass ? lane : 0, step = pass ? 32 : 1;
            int nd = need[b];
            if (nd > 0 && int64_t(start[b]) + nd > found) {
                if (me == 0) atomicOr(&sh.bad, TQ_DEV_NO_PAGES);
                nd = -1;
            }
            if (nd >= 0) {
                reserve_row(a, b, add, nd, start[b], at, slots, me, step);
            } else {                                     // nothing reserved: these tokens are skipped by a write
                for (int64_t t = me; t < add && at + t < n_slots; t += step) slots[at + t] = -1;
            }
        }
    }
    for (int64_t t = first + threadIdx.x; t < n_slots; t += kPlanThreads) slots[t] = -1;
    __syncthreads();
    if (threadIdx.x == 0 && sh.bad) atomicOr(a.ws.status, sh.bad);
}

// ---------------------------------------------------------------------------
// free
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) free_kernel(PoolArgs a, const int32_t *rows, int n) {
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= n) return;
    const int r = rows[i];
    if (r < 0 || r >= a.n_rows) {
        if (lane == 0) atomicOr(a.ws.status, TQ_DEV_ROW);
        return;
    }
    // whoever takes the length frees the row: a row named twice is freed once
    int len = 0;
    if (lane == 0) len = atomicExch(&a.lens[r], 0);
    len = __shfl_sync(kFull, len, 0);
    if (len < 0 || len > a.max_blocks * int64_t(a.P)) {
        if (lane == 0) atomicOr(a.ws.status, TQ_DEV_ROW);
        return;
    }
    const int pages = int((int64_t(len) + a.P - 1) / a.P);
    for (int j = lane; j < pages; j += 32) release(a, a.table[int64_t(r) * a.max_blocks + j]);
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
// What a page of the new row holds: its own tokens at their own positions,
// others, or a token that is not there.
constexpr int kSame = 0, kOthers = 1, kOutOfRange = 2;
__host__ __device__ __forceinline__ int pages_kept(const PoolArgs &a, int keep_stride) {
    const int64_t pages = (int64_t(keep_stride) + a.P - 1) / a.P;
    return int(pages < a.max_blocks ? pages : a.max_blocks);
}
// A warp a page; the lists are what is long here (read by the planning block,
// eight of 4,095 took it 32 of its 43 us).
__global__ void __launch_bounds__(256) compact_look_kernel(PoolArgs a, const int32_t *rows, const int32_t *keep,
                                                           int keep_stride, const int32_t *keep_lens, int n) {
    let_next_in();
    const int lane = threadIdx.x & 31, most = pages_kept(a, keep_stride);
    const int64_t w = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int i = int(w / most), j = int(w - int64_t(i) * most);
    if (i >= n) return;
    const int r = rows[i], kept = min(keep_lens[i], keep_stride);
    if (r < 0 || r >= a.n_rows || j * a.P >= kept) return;
    const int len = a.lens[r], p1 = min(kept, (j + 1) * a.P);
    const int32_t *list = keep + int64_t(i) * keep_stride;
    bool same = true, in = true;
#pragma unroll 2
    for (int p = j * a.P + lane; p < p1; p += 32) {
        const int t = list[p];
        in &= t >= 0 && t < len;
        same &= t == p;
    }
    in = __all_sync(kFull, in);
    same = __all_sync(kFull, same);
    if (lane == 0) a.ws.fresh[int64_t(i) * a.max_blocks + j] = !in ? kOutOfRange : same ? kSame : kOthers;
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(PoolArgs a, const int32_t *rows,
                                                                    int keep_stride, const int32_t *keep_lens, int n) {
    __shared__ PlanShared sh;
    wait_for_last();
    let_next_in();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool few = n <= kSharedRequests;
    // lens: the rows' lengths; out: a kept token is out of range (start's room,
    // which is filled later)
    int32_t *need = few ? sh.need : a.ws.need, *start = few ? sh.start : a.ws.start, *out = start;
    int32_t *lens = few ? sh.len : a.ws.len;
    int32_t *mark = a.n_rows <= kSharedRows ? sh.mark : a.ws.mark;
    if (threadIdx.x == 0) {
        sh.jobs = 0;
        sh.bad = 0;
    }
    mark_rows(a, rows, n, mark);
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int r = rows[i];
        uint32_t bad = 0;
        lens[i] = out[i] = 0;
        if (r < 0 || r >= a.n_rows || mark[r] != i) bad = TQ_DEV_ROW;
        else {
            const int len = a.lens[r], kept = keep_lens[i];
            lens[i] = len;
            if (len < 0 || len > a.max_blocks * int64_t(a.P)) bad = TQ_DEV_ROW;
            else if (kept < 0 || kept > keep_stride) bad = TQ_DEV_KEEP_RANGE;
            else if (kept > a.max_blocks * int64_t(a.P)) bad = TQ_DEV_NO_PAGES;
        }
        need[i] = bad ? -1 : 0;
        if (bad) atomicOr(&sh.bad, bad);
    }
    __syncthreads();
    for (int i = warp; i < n; i += kPlanWarps) {     // the pages as they were
        if (need[i] < 0) continue;
        const int r = rows[i], had = int((int64_t(lens[i]) + a.P - 1) / a.P);
        const int32_t *row = a.table + int64_t(r) * a.max_blocks;
        bool ok = true;
#pragma unroll 4
        for (int j = lane; j < had; j += 32) {
            const int id = row[j];
            a.ws.old[int64_t(i) * a.max_blocks + j] = id;
            ok &= live_page(a, id);
        }
        ok = __all_sync(kFull, ok);
        __syncwarp();
        if (!ok && lane == 0) {
            need[i] = -1;
            atomicOr(&sh.bad, TQ_DEV_BLOCK_RANGE);
        }
    }
    __syncthreads();
    const int most = pages_kept(a, keep_stride);
    for (int64_t w = threadIdx.x; w < int64_t(n) * most; w += kPlanThreads) {
        // a page stays where it keeps its tokens and is full or this row's alone
        const int i = int(w / most), j = int(w - int64_t(i) * most), kept = keep_lens[i];
        if (need[i] < 0 || j * a.P >= kept) continue;
        int32_t *f = a.ws.fresh + int64_t(i) * a.max_blocks + j;
        const int seen = *f;
        if (seen == kOutOfRange) out[i] = 1;
        else
            *f = seen == kSame && ((j + 1) * a.P <= kept || a.refs[a.table[int64_t(rows[i]) * a.max_blocks + j]] == 1) ? -1
                                                                                                                     : 0;
    }
    __syncthreads();
    for (int i = warp; i < n; i += kPlanWarps) {     // ranks of the fresh pages in their request
        if (need[i] < 0) continue;
        const int want = int((int64_t(keep_lens[i]) + a.P - 1) / a.P);
        int32_t *fresh = a.ws.fresh + int64_t(i) * a.max_blocks;
        int rank = 0;
        const bool in = !out[i];
        for (int j0 = 0; j0 < want && in; j0 += 32) {
            const int j = j0 + lane, v = j < want ? fresh[j] : -1;
            const uint32_t dealt = __ballot_sync(kFull, v == 0);
            if (v == 0) fresh[j] = rank + __popc(dealt & ((1u << lane) - 1u));
            rank += __popc(dealt);
        }
        __syncwarp();
        if (lane == 0) {
            need[i] = in ? rank : -1;
            if (!in) atomicOr(&sh.bad, TQ_DEV_KEEP_RANGE);
        }
    }
    __syncthreads();
    const int64_t total = deal_ranks(need, start, n, sh);
    const int found = find_free(a.refs, a.num_blocks, total, a.ws.ids, sh);
    for (int i = warp; i < n; i += kPlanWarps) {
        const int nd = need[i], at = start[i];
        if (nd < 0) continue;
        if (nd > 0 && int64_t(at) + nd > found) {
            if (lane == 0) atomicOr(&sh.bad, TQ_DEV_NO_PAGES);
            continue;
        }
        const int r = rows[i], kept = keep_lens[i];
        const int had = int((int64_t(lens[i]) + a.P - 1) / a.P), want = int((int64_t(kept) + a.P - 1) / a.P);
        int32_t *row = a.table + int64_t(r) * a.max_blocks;
        const int32_t *fresh = a.ws.fresh + int64_t(i) * a.max_blocks;
        const int32_t *old = a.ws.old + int64_t(i) * a.max_blocks;
#pragma unroll 4
        for (int j = lane; j < max(had, want); j += 32) {
            const int rank = j < want ? fresh[j] : 0;
            if (j < had && (j >= want || rank >= 0)) release(a, old[j]);
            if (j < want && rank >= 0) {
                const int id = a.ws.ids[at + rank];
                a.ws.jobs[at + rank] = make_int4(i, j, id, 0);
                row[j] = id;
                a.refs[id] = 1;
            }
        }
        __syncwarp();
        if (lane == 0) {
            if (nd > 0) atomicMax(&sh.jobs, at + nd);  // those served hold the ranks before this
            a.lens[r] = kept;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        *a.ws.n_jobs = sh.jobs;
        if (sh.bad) atomicOr(a.ws.status, sh.bad);
    }
}

struct GatherArgs {
    PlanWs ws;
    const int32_t *keep, *keep_lens;
    int keep_stride, max_blocks, P, H, heads, page_bytes, n_fields;
    int off[12], bpt[12];        // fields of a page: byte offset, bytes per token (a power of two)
    int shift[12];               // log2 of the 16-byte (or smaller) pieces of a token's field
    int first[13];               // first piece of a field among those of 1 << shift per token slot
};

// Copies the records of one fresh page in one layer (blockIdx.y), `heads` heads
// a block.  Where each position's token lies is looked up once, into shared
// memory; then the pieces of all fields, 16 bytes or the whole of a smaller
// field, are one list that the threads share, each for four heads at once (four
// loads in flight).  Bound by DRAM latency and the number of loads in flight:
// a head a block, one field after the other, moved 434 MB in 120 us;
// this takes 94.
constexpr int kGatherThreads = 128, kGatherHeads = 4;
template <typename V>
__device__ __forceinline__ void move4(uint8_t *const (&to)[kGatherHeads], const uint8_t *const (&from)[kGatherHeads], int n) {
    V v[kGatherHeads];
#pragma unroll
    for (int k = 0; k < kGatherHeads; ++k)
        if (k < n) v[k] = *reinterpret_cast<const V *>(from[k]);
#pragma unroll
    for (int k = 0; k < kGatherHeads; ++k)
        if (k < n) *reinterpret_cast<V *>(to[k]) = v[k];
}
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ Layers layers,
                                                                const __grid_constant__ GatherArgs a) {
    __shared__ int64_t from[256];                    // byte of the token's page
    __shared__ int slot[256];                        // and its position there
    wait_for_last();
    const int n_jobs = *a.ws.n_jobs, groups = (a.H + a.heads - 1) / a.heads;
    const int64_t page_stride = int64_t(a.H) * a.page_bytes;
    for (int64_t w = blockIdx.x; w < int64_t(n_jobs) * groups; w += gridDim.x) {
        const int4 job = a.ws.jobs[w / groups];
        const int h0 = int(w % groups) * a.heads, h1 = min(a.H, h0 + a.heads);
        const int cnt = min(a.P, a.keep_lens[job.x] - job.y * a.P);
        const int32_t *list = a.keep + int64_t(job.x) * a.keep_stride + job.y * a.P;
        const int32_t *old = a.ws.old + int64_t(job.x) * a.max_blocks;
        uint8_t *base = layers.at[blockIdx.y];
        __syncthreads();
        for (int p = threadIdx.x; p < cnt; p += kGatherThreads) {
            const int t = list[p], pg = t / a.P;
            from[p] = old[pg] * page_stride;
            slot[p] = t - pg * a.P;
        }
        __syncthreads();
        const int pieces = a.first[a.n_fields] * cnt;
        for (int h = h0; h < h1; h += kGatherHeads)
            for (int u = threadIdx.x; u < pieces; u += kGatherThreads) {
                int f = 0;
                while (u >= a.first[f + 1] * cnt) ++f;
                const int x = u - a.first[f] * cnt, p = x >> a.shift[f], part = (x & ((1 << a.shift[f]) - 1)) * 16;
                const uint8_t *s[kGatherHeads];
                uint8_t *d[kGatherHeads];
#pragma unroll
                for (int k = 0; k < kGatherHeads; ++k) {
                    s[k] = base + from[p] + int64_t(h + k) * a.page_bytes + a.off[f] + slot[p] * a.bpt[f] + part;
                    d[k] = base + job.z * page_stride + int64_t(h + k) * a.page_bytes + a.off[f] + p * a.bpt[f] + part;
                }
                const int n = min(kGatherHeads, h1 - h);
                switch (a.bpt[f]) {
                    case 1: move4<uint8_t>(d, s, n); break;
                    case 2: move4<uint16_t>(d, s, n); break;
                    case 4: move4<uint32_t>(d, s, n); break;
                    case 8: move4<uint2>(d, s, n); break;
                    default: move4<uint4>(d, s, n);
                }
            }
    }
}

Layers layers_of(void *const *caches, int n) {
    Layers ly{};
    for (int i = 0; i < n; ++i) ly.at[i] = static_cast<uint8_t *>(caches[i]);
    return ly;
}

PoolArgs pool_args(const Layout &L, const tq_page_pool &p, uint8_t *ws) {
    PoolArgs a;
    a.refs = p.refs;
    a.table = p.table;
    a.lens = p.lens;
    a.num_blocks = int(p.num_blocks);
    a.max_blocks = p.max_blocks;
    a.n_rows = p.n_rows;
    a.P = L.P;
    carve(ws, p.num_blocks, p.n_rows, p.max_blocks, &a.ws);
    return a;
}

}  // namespace

size_t pages_ws_bytes(int64_t num_blocks, int n_rows, int max_blocks) {
    PlanWs p;
    return carve(nullptr, num_blocks, n_rows, max_blocks, &p);
}

int launch_pages_fork(const Layout &L, const tq_page_pool &pool, void *const *caches, int n_layers, const int32_t *src,
                      const int32_t *dst, int n, uint8_t *ws, void *stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const PoolArgs a = pool_args(L, pool, ws);
    fork_plan_kernel<<<1, kPlanThreads, 0, st>>>(a, src, dst, n);
    const int64_t bytes = int64_t(L.H) * L.page_bytes;
    const unsigned z = unsigned(bytes / 16384 < 1 ? 1 : bytes / 16384 > 64 ? 64 : bytes / 16384);
    for (int l0 = 0; l0 < n_layers; l0 += kLayersPerLaunch) {
        const int nl = n_layers - l0 < kLayersPerLaunch ? n_layers - l0 : kLayersPerLaunch;
        const cudaError_t e = launch_next(copy_pages_kernel, dim3(unsigned(n), unsigned(nl), z), 256, 0, st,
                                          layers_of(caches + l0, nl), a.ws, bytes);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

int launch_pages_reserve(const Layout &L, const tq_page_pool &pool, const int32_t *new_tokens, int32_t *slots,
                         int64_t n_slots, uint8_t *ws, void *stream) {
    reserve_plan_kernel<<<1, kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(pool_args(L, pool, ws), new_tokens,
                                                                                  slots, n_slots);
    return cudaGetLastError();
}

int launch_pages_free(const Layout &L, const tq_page_pool &pool, const int32_t *rows, int n, uint8_t *ws, void *stream) {
    free_kernel<<<unsigned((n + 7) / 8), 256, 0, static_cast<cudaStream_t>(stream)>>>(pool_args(L, pool, ws), rows, n);
    return cudaGetLastError();
}

int launch_pages_compact(const Layout &L, const tq_page_pool &pool, void *const *caches, int n_layers,
                         const int32_t *rows, const int32_t *keep, int keep_stride, const int32_t *keep_lens, int n,
                         uint8_t *ws, void *stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const PoolArgs a = pool_args(L, pool, ws);
    const int64_t lists = (int64_t(n) * pages_kept(a, keep_stride) + 7) / 8;
    if (lists > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaError_t e = cudaSuccess;
    if (lists > 0) {
        compact_look_kernel<<<unsigned(lists), 256, 0, st>>>(a, rows, keep, keep_stride, keep_lens, n);
        e = launch_next(compact_plan_kernel, dim3(1), kPlanThreads, 0, st, a, rows, keep_stride, keep_lens, n);
    } else {
        compact_plan_kernel<<<1, kPlanThreads, 0, st>>>(a, rows, keep_stride, keep_lens, n);
    }
    if (e != cudaSuccess) return e;
    GatherArgs g{};
    g.ws = a.ws;
    g.keep = keep;
    g.keep_lens = keep_lens;
    g.keep_stride = keep_stride;
    g.max_blocks = pool.max_blocks;
    g.P = L.P;
    g.H = L.H;
    g.page_bytes = L.page_bytes;
    auto field = [&](int off, int bpt) {
        if (off < 0) return;
        int shift = 0;
        while ((16 << shift) < bpt) ++shift;
        g.off[g.n_fields] = off;
        g.bpt[g.n_fields] = bpt;
        g.shift[g.n_fields] = shift;
        g.first[g.n_fields + 1] = g.first[g.n_fields] + (1 << shift);
        ++g.n_fields;
    };
    field(L.kc_off, L.kc_bpt);
    field(L.kh_off, L.kh_bpt);
    field(L.kc2_off, L.kc2_bpt);
    field(L.kh2_off, L.kh2_bpt);
    field(L.ks_off, L.ks_bpt);
    field(L.kn_off, 2);
    field(L.kr_off, 2);
    field(L.vc_off, L.vc_bpt);
    field(L.vh_off, L.vh_bpt);
    field(L.vc2_off, L.vc2_bpt);
    field(L.vh2_off, L.vh2_bpt);
    field(L.vn_off, 2);
    // all heads of a page to a block where there are pages enough for some ten
    // blocks an SM, else fewer
    const int64_t pages = int64_t(n) * ((int64_t(keep_stride) + L.P - 1) / L.P);
    int64_t heads = pages * n_layers * L.H / (148 * 10);
    heads = heads < kGatherHeads ? kGatherHeads : heads > L.H ? L.H : heads / kGatherHeads * kGatherHeads;
    g.heads = int(heads);
    const int64_t most = pages * ((L.H + heads - 1) / heads);
    const unsigned x = unsigned(most < 1 ? 1 : most > 65536 ? 65536 : most);
    for (int l0 = 0; l0 < n_layers; l0 += kLayersPerLaunch) {
        const int nl = n_layers - l0 < kLayersPerLaunch ? n_layers - l0 : kLayersPerLaunch;
        e = launch_next(gather_kernel, dim3(x, unsigned(nl)), kGatherThreads, 0, st, layers_of(caches + l0, nl), g);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

}  // namespace tq
