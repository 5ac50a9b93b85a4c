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
    p->slot0 = reinterpret_cast<int64_t *>(take(8 * size_t(n_rows)));
    p->ids = reinterpret_cast<int32_t *>(take(4 * size_t(num_blocks)));
    p->jobs = reinterpret_cast<int4 *>(take(16 * size_t(num_blocks)));
    p->old = reinterpret_cast<int32_t *>(take(4 * size_t(n_rows) * size_t(max_blocks)));
    p->fresh = reinterpret_cast<int32_t *>(take(4 * size_t(n_rows) * size_t(max_blocks)));
    return off;
}

struct PlanShared {
    int64_t part[kPlanWarps];
    int64_t carry;
    int count, jobs;
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
    int64_t before = 0, all = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
        if (w < warp) before += sh.part[w];
        all += sh.part[w];
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

// start[i] = the sum of max(need, 0) before i; returns the sum over all.
__device__ int64_t deal_ranks(const PlanWs &ws, int n, PlanShared &sh) {
    int64_t carry = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        const int64_t v = i < n ? max(ws.need[i], 0) : 0;
        int64_t total;
        const int64_t at = carry + block_scan(v, sh, &total);
        if (i < n) ws.start[i] = int(min(at, int64_t(INT_MAX)));
        carry += total;
    }
    __syncthreads();
    return carry;
}

// The lowest `want` free pages into ids, ascending; returns how many there are.
__device__ int find_free(const int32_t *refs, int num_blocks, int64_t want, int32_t *ids, PlanShared &sh) {
    int found = 0;
    for (int b0 = 0; b0 < num_blocks && found < want; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        const bool is_free = b < num_blocks && refs[b] == 0;
        int64_t total;
        const int at = found + int(block_scan(is_free ? 1 : 0, sh, &total));
        if (is_free && at < want) ids[at] = b;
        found += int(total);
    }
    __syncthreads();
    return int(min(int64_t(found), want));
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
__device__ void mark_rows(const PoolArgs &a, const int32_t *rows, int n) {
    for (int r = threadIdx.x; r < a.n_rows; r += kPlanThreads) a.ws.mark[r] = INT_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        if (rows[i] >= 0 && rows[i] < a.n_rows) atomicMin(&a.ws.mark[rows[i]], i);
    __syncthreads();
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(PoolArgs a, const int32_t *src, const int32_t *dst,
                                                                 int n) {
    __shared__ PlanShared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    mark_rows(a, dst, n);
    for (int i = warp; i < n; i += kPlanWarps) {
        const int s = src[i], d = dst[i];
        uint32_t bad = 0;
        if (s < 0 || s >= a.n_rows || d < 0 || d >= a.n_rows || a.ws.mark[d] != i || a.lens[d] != 0)
            bad = TQ_DEV_ROW;
        else if (a.lens[s] < 0 || a.lens[s] > a.max_blocks * int64_t(a.P))
            bad = TQ_DEV_ROW;
        int need = -1;
        if (!bad) {
            const int len = a.lens[s], pages = int((int64_t(len) + a.P - 1) / a.P);
            bool ok = true;
            for (int j = lane; j < pages; j += 32) ok = ok && live_page(a, a.table[int64_t(s) * a.max_blocks + j]);
            if (!__all_sync(kFull, ok)) bad = TQ_DEV_BLOCK_RANGE;
            else need = len % a.P != 0;
        }
        if (lane == 0) {
            a.ws.need[i] = need;
            // the length is read here: rows that a later phase fills are empty now
            a.ws.old[i] = need >= 0 ? a.lens[s] : 0;
            if (bad) atomicOr(a.ws.status, bad);
        }
    }
    __syncthreads();
    const int64_t want = deal_ranks(a.ws, n, sh);
    const int found = find_free(a.refs, a.num_blocks, want, a.ws.ids, sh);
    for (int i = warp; i < n; i += kPlanWarps) {
        const int need = a.ws.need[i], at = a.ws.start[i];
        if (need < 0) continue;
        if (need > 0 && at >= found) {
            if (lane == 0) atomicOr(a.ws.status, TQ_DEV_NO_PAGES);
            continue;
        }
        const int len = a.ws.old[i], full = len / a.P;
        const int32_t *from = a.table + int64_t(src[i]) * a.max_blocks;
        int32_t *to = a.table + int64_t(dst[i]) * a.max_blocks;
        for (int j = lane; j < full; j += 32) {
            const int id = from[j];
            to[j] = id;
            atomicAdd(&a.refs[id], 1);
        }
        if (lane == 0) {
            if (need) {
                const int id = a.ws.ids[at];
                a.ws.jobs[at] = make_int4(from[full], id, 0, 0);
                to[full] = id;
                a.refs[id] = 1;
            }
            a.lens[dst[i]] = len;
        }
    }
    if (threadIdx.x == 0) *a.ws.n_jobs = found;      // one page a request: every page found is dealt
}

// The layers' cache addresses travel as a kernel argument (1 KB a launch).
constexpr int kLayersPerLaunch = 128;
struct Layers {
    uint8_t *at[kLayersPerLaunch];
};

// Job's page copied in layer blockIdx.y; blockIdx.z takes a slice of it.
__global__ void __launch_bounds__(256) copy_pages_kernel(const __grid_constant__ Layers layers, PlanWs ws,
                                                         int64_t block_bytes) {
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
__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(PoolArgs a, const int32_t *new_tokens,
                                                                    int32_t *slots, int64_t n_slots) {
    __shared__ PlanShared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t first = 0;                                   // entries of slot_mapping before this chunk of rows
    for (int b0 = 0; b0 < a.n_rows; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        const int64_t add = b < a.n_rows ? max(new_tokens[b], 0) : 0;
        int64_t total;
        const int64_t at = first + block_scan(add, sh, &total);
        first += total;
        if (b >= a.n_rows) continue;
        int need = -1;
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
            if (bad) atomicOr(a.ws.status, bad);
            else need = int(then - pages);
        }
        a.ws.need[b] = need;
        a.ws.slot0[b] = at;
    }
    __syncthreads();
    const int64_t want = deal_ranks(a.ws, a.n_rows, sh);
    const int found = find_free(a.refs, a.num_blocks, want, a.ws.ids, sh);
    for (int b = warp; b < a.n_rows; b += kPlanWarps) {
        const int64_t add = max(new_tokens[b], 0), at = a.ws.slot0[b];
        int need = a.ws.need[b];
        const int rank = a.ws.start[b];
        if (need > 0 && int64_t(rank) + need > found) {
            if (lane == 0) atomicOr(a.ws.status, TQ_DEV_NO_PAGES);
            need = -1;
        }
        if (need < 0) {                                  // nothing reserved: these tokens are skipped by a write
            for (int64_t t = lane; t < add && at + t < n_slots; t += 32) slots[at + t] = -1;
            continue;
        }
        const int64_t len = a.lens[b];
        const int pages = int((len + a.P - 1) / a.P);
        int32_t *row = a.table + int64_t(b) * a.max_blocks;
        for (int j = lane; j < need; j += 32) {
            const int id = a.ws.ids[rank + j];
            row[pages + j] = id;
            a.refs[id] = 1;
        }
        __syncwarp();
        for (int64_t t = lane; t < add; t += 32) {
            const int64_t pos = len + t;
            slots[at + t] = row[pos / a.P] * a.P + int(pos % a.P);
        }
        __syncwarp();
        if (lane == 0) a.lens[b] = int(len + add);
    }
    for (int64_t t = first + threadIdx.x; t < n_slots; t += kPlanThreads) slots[t] = -1;
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
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(PoolArgs a, const int32_t *rows,
                                                                    const int32_t *keep, int keep_stride,
                                                                    const int32_t *keep_lens, int n) {
    __shared__ PlanShared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) sh.jobs = 0;
    mark_rows(a, rows, n);
    for (int i = warp; i < n; i += kPlanWarps) {
        const int r = rows[i];
        uint32_t bad = 0;
        int len = 0, kept = 0;
        if (r < 0 || r >= a.n_rows || a.ws.mark[r] != i) bad = TQ_DEV_ROW;
        else {
            len = a.lens[r];
            kept = keep_lens[i];
            if (len < 0 || len > a.max_blocks * int64_t(a.P)) bad = TQ_DEV_ROW;
            else if (kept < 0 || kept > keep_stride) bad = TQ_DEV_KEEP_RANGE;
            else if (kept > a.max_blocks * int64_t(a.P)) bad = TQ_DEV_NO_PAGES;
        }
        const int32_t *list = keep + int64_t(i) * keep_stride;
        const int32_t *row = a.table + int64_t(r) * a.max_blocks;
        int need = 0;
        if (!bad) {
            const int had = int((int64_t(len) + a.P - 1) / a.P), want = int((int64_t(kept) + a.P - 1) / a.P);
            bool ok = true;
            for (int j = lane; j < had; j += 32) {
                const int id = row[j];
                a.ws.old[int64_t(i) * a.max_blocks + j] = id;
                ok = ok && live_page(a, id);
            }
            if (!__all_sync(kFull, ok)) bad = TQ_DEV_BLOCK_RANGE;
            for (int j = 0; j < want && !bad; ++j) {
                // a page stays where every position keeps its own token, and
                // it is either full or this row's alone
                bool same = true, in = true;
                const int p1 = min(kept, (j + 1) * a.P);
                for (int p = j * a.P + lane; p < p1; p += 32) {
                    const int t = list[p];
                    in = in && t >= 0 && t < len;
                    same = same && t == p;
                }
                if (!__all_sync(kFull, in)) { bad = TQ_DEV_KEEP_RANGE; break; }
                same = __all_sync(kFull, same);
                const bool stays = same && (p1 == (j + 1) * a.P || a.refs[row[j]] == 1);
                if (lane == 0) a.ws.fresh[int64_t(i) * a.max_blocks + j] = stays ? -1 : need;
                if (!stays) ++need;
            }
        }
        if (lane == 0) {
            a.ws.need[i] = bad ? -1 : need;
            if (bad) atomicOr(a.ws.status, bad);
        }
    }
    __syncthreads();
    const int64_t total = deal_ranks(a.ws, n, sh);
    const int found = find_free(a.refs, a.num_blocks, total, a.ws.ids, sh);
    for (int i = warp; i < n; i += kPlanWarps) {
        const int need = a.ws.need[i], at = a.ws.start[i];
        if (need < 0) continue;
        if (need > 0 && int64_t(at) + need > found) {
            if (lane == 0) atomicOr(a.ws.status, TQ_DEV_NO_PAGES);
            continue;
        }
        const int r = rows[i], len = a.lens[r], kept = keep_lens[i];
        const int had = (len + a.P - 1) / a.P, want = (kept + a.P - 1) / a.P;
        int32_t *row = a.table + int64_t(r) * a.max_blocks;
        const int32_t *fresh = a.ws.fresh + int64_t(i) * a.max_blocks;
        const int32_t *old = a.ws.old + int64_t(i) * a.max_blocks;
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
        if (lane == 0) {
            if (need > 0) atomicMax(&sh.jobs, at + need);  // those served hold the ranks before this
            a.lens[r] = kept;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) *a.ws.n_jobs = sh.jobs;
}

struct GatherArgs {
    PlanWs ws;
    const int32_t *keep, *keep_lens;
    int keep_stride, max_blocks, P, H, page_bytes, n_fields;
    int off[12], bpt[12];        // fields of a page: byte offset, bytes per token (a power of two)
};

// Copies the records of one fresh page of one head in one layer (blockIdx.y):
// thread (position, unit of up to 16 bytes) per field.
__global__ void __launch_bounds__(128) gather_kernel(const __grid_constant__ Layers layers, GatherArgs a) {
    const int n_jobs = *a.ws.n_jobs;
    const int64_t page_stride = int64_t(a.H) * a.page_bytes;
    for (int64_t w = blockIdx.x; w < int64_t(n_jobs) * a.H; w += gridDim.x) {
        const int4 job = a.ws.jobs[w / a.H];
        const int h = int(w % a.H);
        const int cnt = min(a.P, a.keep_lens[job.x] - job.y * a.P);
        const int32_t *list = a.keep + int64_t(job.x) * a.keep_stride + job.y * a.P;
        const int32_t *old = a.ws.old + int64_t(job.x) * a.max_blocks;
        uint8_t *base = layers.at[blockIdx.y] + int64_t(h) * a.page_bytes;
        uint8_t *to = base + job.z * page_stride;
        for (int f = 0; f < a.n_fields; ++f) {
            const int bpt = a.bpt[f], unit = min(bpt, 16), per = bpt / unit;
            for (int u = threadIdx.x; u < cnt * per; u += 128) {
                const int p = u / per, part = u % per;
                const int t = list[p];
                const uint8_t *s = base + old[t / a.P] * page_stride + a.off[f] + (t % a.P) * bpt + part * unit;
                uint8_t *d = to + a.off[f] + p * bpt + part * unit;
                switch (unit) {
                    case 16: *reinterpret_cast<uint4 *>(d) = *reinterpret_cast<const uint4 *>(s); break;
                    case 8: *reinterpret_cast<uint2 *>(d) = *reinterpret_cast<const uint2 *>(s); break;
                    case 4: *reinterpret_cast<uint32_t *>(d) = *reinterpret_cast<const uint32_t *>(s); break;
                    case 2: *reinterpret_cast<uint16_t *>(d) = *reinterpret_cast<const uint16_t *>(s); break;
                    default: *d = *s;
                }
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
        copy_pages_kernel<<<dim3(unsigned(n), unsigned(nl), z), 256, 0, st>>>(layers_of(caches + l0, nl), a.ws, bytes);
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
    compact_plan_kernel<<<1, kPlanThreads, 0, st>>>(a, rows, keep, keep_stride, keep_lens, n);
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
        g.off[g.n_fields] = off;
        g.bpt[g.n_fields++] = bpt;
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
    const int64_t most = int64_t(n) * ((keep_stride + L.P - 1) / L.P) * L.H;
    const unsigned x = unsigned(most < 1 ? 1 : most > 65536 ? 65536 : most);
    for (int l0 = 0; l0 < n_layers; l0 += kLayersPerLaunch) {
        const int nl = n_layers - l0 < kLayersPerLaunch ? n_layers - l0 : kLayersPerLaunch;
        gather_kernel<<<dim3(x, unsigned(nl)), 128, 0, st>>>(layers_of(caches + l0, nl), g);
    }
    return cudaGetLastError();
}

}  // namespace tq
