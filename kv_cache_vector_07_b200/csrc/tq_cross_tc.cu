// Cross attention on the tensor cores, for head sizes 64 and 128 under the
// Hadamard rotation, any codec, any page size.
//
//   k_t = nhat_t c[code_t] + rho_t sqrt(pi/2)/m S^T (2 s_t - 1),  v_t = nhat_v,t c_v[code_v,t]
//   o   = R_v^T sum_t softmax_t(<R q, k_t> / sqrt(d)) v_t
//
// Every query of a run reads the same states, so they are decoded once:
//
//   expand   128 tokens of one KV head at a time: k_t and v_t in their rotated
//            bases as fp16 operand tiles in the workspace, laid out as the
//            tensor cores read them from shared memory.  S^T s is a product of
//            +-1 signs (exact) with S as fp16 (exact for |S| >= 2^-14) on
//            tcgen05.  A tile is scaled by a power of two that brings a bound on
//            its coordinates (from its largest norm) to [2^14, 2^15), so states
//            of any norm keep fp16's 11 bits down to 2^-28 of that bound.
//   attend   256 query rows (two tiles of 128 rows: positions x heads of the
//            group) walk the tiles: S = Q K^T and O += P V on tcgen05, the
//            online softmax between them, a thread per row.
//
// Queries are rotated and scaled to fp16 as they are staged (the same range),
// softmax weights are fp16, all sums fp32: queries and states are off by at
// most 2^-11 of themselves, eight times finer than the bf16 result.  The tile
// scales ride along for nothing: the key's on the factor that turns S into a
// logarithm, the value's (2^e) on its offset, P' = 2^(l + e - m), while the sum
// takes P' 2^-e.  The reference m follows l + e at a distance that keeps the
// strongest weight of every tile between 2^-9 and 2^15: a weight is off by at
// most 2^-11 of itself or 2^-25, half the smallest step of fp16, which is 2^-16
// of its tile's strongest at worst and 2^-32 of the one that set m.  Keys whose
// value is zero are left out of all this, however strong they are: their weights
// go to the sum alone, in fp32.
#include <atomic>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "tc05.cuh"
#include "tq_chain.cuh"
#include "tq_dev.cuh"

namespace tq {
namespace {

constexpr int kTile = 128;                 // keys of a tile, and query rows of one

// What the attention needs of a tile beside its operands.
struct __align__(16) TileMeta {
    float kscale;                          // key = stored * kscale
    float vexp, vinv;                      // value = stored * 2^vexp; vinv = 2^-vexp
    uint32_t has_zero;                     // a bit of zero is set
    uint32_t mask[4];                      // key k of the tile is there, and its value is not zero
    uint32_t zero[4];                      // it is there, and its value is zero
};

constexpr size_t image_bytes(int d) { return size_t(kTile) * d * 2; }   // one operand tile

__device__ __forceinline__ uint32_t h2u(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Packed pairs of fp32 (one issue slot for two operations).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                 "r"(tc05::smem_u32(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Bounded wait: about a second.
__device__ __forceinline__ bool wait_bounded(uint64_t *bar, uint32_t parity) {
    for (uint32_t i = 0; i < 500000u; ++i)
        if (tc05::mbar_try_wait_sleep(bar, parity, 2000u)) return true;
    return false;
}

// Bounded wait (a second or more) that also gives up once another thread has.
// The first polls name no time to sleep: a thread woken from a long sleep
// came back some 500 cycles late.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile uint32_t *abort_flag) {
    for (uint32_t i = 0; i < 256u; ++i)
        if (tc05::mbar_test_wait(bar, parity)) return true;
    for (uint32_t i = 0; i < 500000u; ++i) {
        if (tc05::mbar_try_wait_sleep(bar, parity, 2000u)) return true;
        if ((i & 63u) == 63u && *abort_flag) return false;
    }
    *abort_flag = 1u;
    return false;
}

// ---------------------------------------------------------------------------
// expand
// ---------------------------------------------------------------------------
struct ExpandArgs {
    Layout L;
    DevParams kp, vp;
    const int32_t *table, *kv_lens;
    int bt_stride, max_kv_len;
    const uint8_t *cache;
    int64_t num_blocks;
    int pair0, n_pairs, n_tiles;           // pairs (sequence, KV head) of this launch
    int32_t *order;                        // [n_pairs] see order_pairs
    int B;
    uint8_t *images;                       // [pair][tile][keys | values]
    TileMeta *meta;                        // [pair][tile]
    uint32_t *status;
};

// A thread's half of a token's codes (keys or values): where they are and how
// wide.  A fractional rate has an array and a codebook for each half.
struct HalfCode {
    int off, bpt, hoff, hbpt;              // array of fields, 3-bit codes' sign bits
    int width;                             // 1, 2, 4 bits; 8: E4M3; 0: polar
    bool signs;
    const float *lv;                       // levels by code (shared memory)
};

// The bytes of the thread's D / 2 codes of up to 4 bits, as they lie in the
// page, and a 3-bit code's sign bits.
template <int D>
struct HalfBytes {
    uint32_t w[D / 16], sg[D / 64];
};
template <int D>
__device__ __forceinline__ void fetch_codes(const HalfCode &hc, const uint8_t *page, int pos, HalfBytes<D> &v) {
    const uint8_t *at = page + hc.off + pos * hc.bpt;
    auto vec = [&](int i) {                            // 16 bytes
        const uint4 u = reinterpret_cast<const uint4 *>(at)[i];
        v.w[4 * i] = u.x; v.w[4 * i + 1] = u.y; v.w[4 * i + 2] = u.z; v.w[4 * i + 3] = u.w;
    };
    if (hc.width == 4) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) vec(i);
    } else if (hc.width == 2) {
        if constexpr (D == 128) {
            vec(0);
        } else {
            v.w[0] = reinterpret_cast<const uint32_t *>(at)[0];
            v.w[1] = reinterpret_cast<const uint32_t *>(at)[1];
        }
    } else if (hc.width == 1) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) v.w[i] = reinterpret_cast<const uint32_t *>(at)[i];
    }
    if (hc.signs) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) v.sg[i] = reinterpret_cast<const uint32_t *>(page + hc.hoff + pos * hc.hbpt)[i];
    }
}

// chunk(c, y) for the thread's coordinates, eight at a time, without their norm.
template <int D, int W, bool SIGNS, typename F>
__device__ __forceinline__ void walk_codes(const HalfCode &hc, const HalfBytes<D> &v, F &&chunk) {
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = c * 8 + e;
            uint32_t k = (v.w[i * W / 32] >> (i * W % 32)) & ((1u << W) - 1u);
            if (SIGNS) k |= ((v.sg[i >> 5] >> (i & 31)) & 1u) << 2;
            y[e] = hc.lv[k];
        }
        chunk(c, y);
    }
}
template <int D, typename F>
__device__ __forceinline__ void walk(const HalfCode &hc, const HalfBytes<D> &v, const uint8_t *page, int pos, int hh,
                                     int off2, int bpt2, const float *polar, F &&chunk) {
    switch (hc.width) {
        case 4: walk_codes<D, 4, false>(hc, v, chunk); break;
        case 2:
            if (hc.signs) walk_codes<D, 2, true>(hc, v, chunk);
            else walk_codes<D, 2, false>(hc, v, chunk);
            break;
        case 1: walk_codes<D, 1, false>(hc, v, chunk); break;
        case 8:                                        // E4M3 bytes, read here
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                const uint2 u = reinterpret_cast<const uint2 *>(page + hc.off + pos * hc.bpt)[c];
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = e4m3_to_float(uint8_t((e < 4 ? u.x : u.y) >> (8 * (e & 3))));
                chunk(c, y);
            }
            break;
        default:
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                float y[8];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const float2 u = polar_pair<D>(page + hc.off + pos * hc.bpt, page + off2 + pos * bpt2, polar,
                                                   hh * (D / 4) + 4 * c + p);
                    y[2 * p] = u.x;
                    y[2 * p + 1] = u.y;
                }
                chunk(c, y);
            }
    }
}

template <int D>
constexpr size_t expand_smem() { return size_t(D) * D * 2 + 2 * image_bytes(D) + 1024; }

// Power of two that brings mx to [2^(top - 1), 2^top); *e: value = stored * 2^e.
// The factor ends at 2^127: what is smaller than 2^(top - 128) (tiny queries)
// stays below 2^(top - 1).
__device__ __forceinline__ float scale_to(float mx, int top, int *e) {
    int ex = top;
    if (mx > 0.f && mx < INFINITY) frexpf(mx, &ex);
    ex = max(ex, top - 127);
    *e = ex - top;
    return ldexpf(1.f, top - ex);
}

// The pairs of the launch, those of long sequences first, for the attention's
// blocks: with the longest last, their blocks run on alone (8 runs of 1,024
// over 1 to 8,192 states, counted out over 148 SMs: 204 steps of a tile until
// the last SM is done unsorted, 188 sorted).  Ranks by counting, up to
// kMaxOrder sequences (there are enough blocks to even out beyond that) and
// only where one launch has every pair.
constexpr int kMaxOrder = 512;
__device__ void order_pairs(const ExpandArgs &a) {
    const bool sort = a.B <= kMaxOrder && a.n_pairs == a.B * a.L.H;
    for (int p = threadIdx.x; p < a.n_pairs; p += blockDim.x) {
        int to = p;
        if (sort) {
            const int b = p / a.L.H, len = a.kv_lens[b];
            int before = 0;
            for (int c = 0; c < a.B; ++c) before += a.kv_lens[c] > len || (a.kv_lens[c] == len && c < b);
            to = before * a.L.H + p % a.L.H;
        }
        a.order[to] = p;
    }
}

// Persistent over (pair, tile); 256 threads, thread (key, half of its
// coordinates): one table lookup and a product a value, one more for a key's
// sketch.  (Kept in fp32 registers until the tile's true maximum was known, and
// with the codec looked at in every chunk, it took four times the
// instructions: 130 us for 2,240 tiles at d = 128, which now take 72.)  Bound by
// the loads of the next item, which the fences between the stages of this one
// wait for: 3,000 to 5,000 of an item's 12,000 cycles.
template <int D>
__global__ void __launch_bounds__(256, 2) cross_expand_kernel(const __grid_constant__ ExpandArgs a) {
    constexpr int HALF = D / 2, NC = D / 16;          // coordinates and 16-byte chunks of a thread
    constexpr uint32_t kImg = uint32_t(image_bytes(D));
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_holder;
    __shared__ __align__(8) uint64_t bar;
    __shared__ float red[2][2][8];
    __shared__ uint32_t red_zero[2][8];
    __shared__ float lv[4][16], polar[2][132];
    __shared__ float bound[2];                        // of a coordinate over the vector's norm
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sS = sm, *sK = sm + D * D * 2, *sV = sK + kImg;
    const Layout &L = a.L;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int key = tid & 127, hh = tid >> 7;

    let_next_in();
    if (blockIdx.x == 0) order_pairs(a);
    // S as the B operand: row j holds S[j][0 .. D), 64 columns to a half
    if (L.kqjl) {
        constexpr int PER = D * D / 8 / 256;              // pieces of a thread, all asked for at once
        uint4 v[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) v[k] = reinterpret_cast<const uint4 *>(a.kp.S16)[k * 256 + tid];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = k * 256 + tid, j = i / (D / 8), c = i % (D / 8);
            *reinterpret_cast<uint4 *>(sS + (c >> 3) * (D * 128) + tc05::sw128_offset(uint32_t(j), uint32_t(c & 7))) = v[k];
        }
    }
    // levels: keys' first and second codebook, values' first and second
    if (tid < 64) {
        const int i = tid & 15, which = tid >> 4;
        const DevParams &P = which < 2 ? a.kp : a.vp;
        const int bits = which == 0 ? L.ka_bits : which == 1 ? L.kb_bits : which == 2 ? L.va_bits : L.vb_bits;
        const float *src = (which & 1) ? ((which == 1 ? L.khalf : L.vhalf) ? P.lv2 : nullptr) : bits <= 4 ? P.lv : nullptr;
        lv[which][i] = src && i < (1 << bits) ? src[i] : 0.f;
    }
    for (int i = tid; i < 132; i += 256) {
        polar[0][i] = L.kpolar ? a.kp.polar[i] : 0.f;
        polar[1][i] = L.vpolar ? a.vp.polar[i] : 0.f;
    }
    if (warp == 0) {
        tc05::tmem_alloc(&tmem_holder, D);
        tc05::tmem_relinquish();
        if (lane == 0) {
            tc05::mbar_init(&bar, 1);
            tc05::fence_mbar_init();
        }
    }
    tc05::fence_proxy_async_smem();
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    if (warp < 2) {
        float mx = warp_max(fabsf(lv[2 * warp + (lane >> 4)][lane & 15]));
        if (warp == 0 && L.kbits == 8) mx = 448.f * rsqrtf(float(D));
        if (warp == 0 ? L.kpolar : L.vpolar) mx = 1.f;
        if (lane == 0) bound[warp] = mx;
    }
    __syncthreads();
    const uint32_t tmem = tmem_holder, lrow = uint32_t((warp & 3) * 32) << 16;
    const float cq = 1.2533141373155003f / float(D);   // sqrt(pi/2) / m
    const bool k2 = L.khalf && hh, v2 = L.vhalf && hh; // this half has arrays of its own
    HalfCode kc, vc;
    kc.width = L.kpolar ? 0 : k2 ? L.kc2_w : L.kc_w;
    kc.off = k2 ? L.kc2_off : L.kc_off + (L.khalf || L.kpolar ? 0 : hh * HALF * L.kc_w / 8);
    kc.bpt = k2 ? L.kc2_bpt : L.kc_bpt;
    kc.signs = (k2 ? L.kb_bits : L.ka_bits) == 3;
    kc.hoff = k2 ? L.kh2_off : L.kh_off + (L.khalf ? 0 : hh * HALF / 8);
    kc.hbpt = k2 ? L.kh2_bpt : L.kh_bpt;
    kc.lv = lv[k2 ? 1 : 0];
    vc.width = L.vpolar ? 0 : v2 ? L.vc2_w : L.vc_w;
    vc.off = v2 ? L.vc2_off : L.vc_off + (L.vhalf || L.vpolar ? 0 : hh * HALF * L.vc_w / 8);
    vc.bpt = v2 ? L.vc2_bpt : L.vc_bpt;
    vc.signs = (v2 ? L.vb_bits : L.va_bits) == 3;
    vc.hoff = v2 ? L.vh2_off : L.vh_off + (L.vhalf ? 0 : hh * HALF / 8);
    vc.hbpt = v2 ? L.vh2_bpt : L.vh_bpt;
    vc.lv = lv[v2 ? 3 : 2];
    uint32_t phase = 0;
    bool timeout = false;

    // Three items are on their way at once: where this thread's key of an item
    // lies is looked up two items ahead, its norms, signs and codes are loaded
    // one ahead (one round of loads after another took 8,000 of an item's
    // 15,000 cycles)
    struct Place {
        bool item;                                     // there is such an item
        int blk, pos, h;                               // pos -1: the key is behind the sequence
        unsigned image;                                // the tile's place in images and meta
    };
    struct Raw {
        Place at;
        const uint8_t *page;                           // null: the key is absent
        uint16_t nk, nv, rk;
        uint32_t sign[D / 64];
        HalfBytes<D> k, v;
    };
    // Items are the tiles that there are, sequence after sequence: seq holds the
    // one that the last item asked for lies in, before_seq the items before it
    // (not every tile of every sequence's room: stepping over the empty ones of
    // short sequences costs a lookup each).
    const int last = a.pair0 + a.n_pairs;
    int seq = a.pair0 / L.H, seq_len = 0, seq_tiles = 0, seq_first = a.pair0;
    unsigned before_seq = 0, seq_items = 0;
    auto enter = [&](int b) {                          // sequence b and its pairs in this launch
        seq = b;
        seq_first = max(a.pair0, b * L.H);
        const int pairs = min(last, (b + 1) * L.H) - seq_first;
        if (pairs <= 0) return false;
        seq_len = min(max(a.kv_lens[b], 0), a.max_kv_len);
        seq_tiles = (seq_len + kTile - 1) / kTile;
        seq_items = unsigned(pairs) * unsigned(seq_tiles);
        return true;
    };
    bool more = enter(seq);
    auto place = [&](unsigned item) {
        Place p{false, -1, -1, 0, 0u};
        while (more && item - before_seq >= seq_items) {
            before_seq += seq_items;
            more = enter(seq + 1);
        }
        if (!more) return p;
        const int within = int(item - before_seq), q = within / seq_tiles, tile = within - q * seq_tiles;
        const int pair = seq_first + q;
        const int t = tile * kTile + key, pg = t / L.P;
        p.item = true;
        p.h = pair - seq * L.H;
        p.image = unsigned(pair - a.pair0) * unsigned(a.n_tiles) + unsigned(tile);
        if (t < seq_len) {
            p.pos = t - pg * L.P;
            p.blk = a.table[int64_t(seq) * a.bt_stride + pg];   // looked at an item later
        }
        return p;
    };
    auto fetch = [&](const Place &at) {
        Raw r;
        r.at = at;
        r.page = nullptr;
        r.nk = r.nv = r.rk = 0;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) r.sign[i] = 0u;
        if (at.blk >= 0 && at.blk < a.num_blocks) {
            const uint8_t *page = a.cache + (int64_t(at.blk) * L.H + at.h) * int64_t(L.page_bytes);
            r.page = page;
            r.nk = *reinterpret_cast<const uint16_t *>(page + L.kn_off + at.pos * 2);
            r.nv = *reinterpret_cast<const uint16_t *>(page + L.vn_off + at.pos * 2);
            if (L.kqjl) {
                r.rk = *reinterpret_cast<const uint16_t *>(page + L.kr_off + at.pos * 2);
#pragma unroll
                for (int i = 0; i < D / 64; ++i)
                    r.sign[i] = reinterpret_cast<const uint32_t *>(page + L.ks_off + at.pos * L.ks_bpt + hh * (HALF / 8))[i];
            }
            fetch_codes<D>(kc, page, at.pos, r.k);
            fetch_codes<D>(vc, page, at.pos, r.v);
        } else if (at.pos >= 0) {
            atomicOr(a.status, TQ_DEV_BLOCK_RANGE);
        }
        return r;
    };
    Raw coming = fetch(place(blockIdx.x));
    Place ahead = place(blockIdx.x + gridDim.x);
    for (unsigned item = blockIdx.x; coming.at.item && !timeout; item += gridDim.x) {
        const Raw raw = coming;
        coming = fetch(ahead);
        ahead = place(item + 2 * gridDim.x);
        const int pos = raw.at.pos;
        const uint8_t *page = raw.page;
        const float nk = h2f_bits(raw.nk), nv = h2f_bits(raw.nv), rk = cq * h2f_bits(raw.rk);
        if (tid == 0) bulk_wait_read();                // the tiles of the item before have been read
        // a key's coordinate is below bound nk + rk sum_j |S_ji|, and |S_ji| below
        // 8.6 (Box-Muller of 53-bit uniforms)
        const float kmx = warp_max(fmaf(fabsf(rk), 8.6f * D, fabsf(nk) * bound[0])), vmx = warp_max(fabsf(nv) * bound[1]);
        const uint32_t none = __ballot_sync(kFull, page && nv == 0.f);
        if (lane == 0) {
            red[0][phase & 1][warp] = kmx;
            red[1][phase & 1][warp] = vmx;
            red_zero[phase & 1][warp] = none;
        }
        __syncthreads();
        float km = 0.f, vm = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            km = fmaxf(km, red[0][phase & 1][i]);
            vm = fmaxf(vm, red[1][phase & 1][i]);
        }
        if (tid == 0) {
            uint32_t any = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) any |= red_zero[phase & 1][i];   // the other warps have the same keys
            a.meta[raw.at.image].has_zero = any;
        }
        int ek, ev;
        const float ksc = scale_to(km, 15, &ek), vsc = scale_to(vm, 15, &ev);
        auto at = [&](uint8_t *img, int c) {           // the thread's chunk c of its key's row
            const int cc = hh * NC + c;
            return reinterpret_cast<uint4 *>(img + (cc >> 3) * 16384 + tc05::sw128_offset(uint32_t(key), uint32_t(cc & 7)));
        };
        if (L.kqjl) {
#pragma unroll
            for (int c = 0; c < NC; c += 4) {
                const uint32_t bits = raw.sign[c / 4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t w[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {      // +1 where the bit is set, else -1 (a missing key's row is not used)
                        const uint32_t u = bits >> (8 * k + 2 * q);
                        w[q] = 0xBC00BC00u ^ (((u << 15) & 0x8000u) | ((u << 30) & 0x80000000u));
                    }
                    *at(sK, c + k) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            tc05::fence_proxy_async_smem();
            tc05::fence_before_sync();
            __syncthreads();
            if (tid == 0) {
                tc05::fence_after_sync();
                constexpr uint32_t idesc = tc05::idesc_f16_f32(128, D) | tc05::kIdescBMajorMN;
                const uint32_t A = tc05::smem_u32(sK), B = tc05::smem_u32(sS);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc05::mma_f16(tmem, tc05::desc_kmajor_sw128(A + uint32_t(ks >> 2) * 16384u + uint32_t(ks & 3) * 32u),
                                  tc05::desc_mnmajor_sw128(B + uint32_t(ks) * 2048u, uint32_t(D) * 128u, 1024u), idesc,
                                  ks > 0);
                tc05::mma_commit(&bar);
            }
        }
        // values, while the product runs
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        if (page) {
            const float f = nv * vsc;
            walk<D>(vc, raw.v, page, pos, hh, L.vc2_off, L.vc2_bpt, polar[1], [&](int c, const float (&y)[8]) {
                *at(sV, c) = make_uint4(h2u(y[0] * f, y[1] * f), h2u(y[2] * f, y[3] * f), h2u(y[4] * f, y[5] * f),
                                        h2u(y[6] * f, y[7] * f));
            });
        } else {
#pragma unroll
            for (int c = 0; c < NC; ++c) *at(sV, c) = zero;
        }
        bool ok = true;
        if (L.kqjl) {
            ok = __all_sync(kFull, wait_bounded(&bar, phase & 1u));
            tc05::fence_after_sync();
        }
        ++phase;
        // keys
        uint32_t r[HALF];
        if (L.kqjl) {
#pragma unroll
            for (int c = 0; c < HALF / 32; ++c)
                tc05::tmem_ld_32x32b_x32(tmem + lrow + uint32_t(hh * HALF + c * 32), reinterpret_cast<uint32_t(&)[32]>(r[c * 32]));
            tc05::tmem_wait_ld();
        } else {
#pragma unroll
            for (int i = 0; i < HALF; ++i) r[i] = 0u;
        }
        if (page) {
            const float f = nk * ksc * (L.kbits == 8 ? rsqrtf(float(D)) : 1.f), g = rk * ksc;
            walk<D>(kc, raw.k, page, pos, hh, L.kc2_off, L.kc2_bpt, polar[0], [&](int c, const float (&y)[8]) {
                float k[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) k[e] = fmaf(g, __uint_as_float(r[c * 8 + e]), y[e] * f);
                *at(sK, c) = make_uint4(h2u(k[0], k[1]), h2u(k[2], k[3]), h2u(k[4], k[5]), h2u(k[6], k[7]));
            });
        } else {
#pragma unroll
            for (int c = 0; c < NC; ++c) *at(sK, c) = zero;
        }
        const uint32_t there = __ballot_sync(kFull, page && nv != 0.f), zero_keys = __ballot_sync(kFull, page && nv == 0.f);
        TileMeta *m = a.meta + raw.at.image;
        if (hh == 0 && lane == 0) {
            m->mask[warp] = there;
            m->zero[warp] = zero_keys;
        }
        if (tid == 0) {
            m->kscale = ldexpf(1.f, ek);
            m->vexp = float(ev);
            m->vinv = ldexpf(1.f, -ev);
        }
        tc05::fence_proxy_async_smem();
        tc05::fence_before_sync();
        timeout = __syncthreads_or(!ok);               // also: every thread has its part of the product
        if (tid == 0 && !timeout) {
            bulk_s2g(a.images + size_t(raw.at.image) * 2 * kImg, sK, 2 * kImg);   // keys, then values
            bulk_commit();
        }
    }
    if (tid == 0) {
        bulk_wait();
        if (timeout) atomicOr(a.status, TQ_DEV_WAIT_TIMEOUT);
    }
    tc05::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc05::fence_after_sync();
        tc05::tmem_dealloc(tmem, D);
    }
}

// ---------------------------------------------------------------------------
// attend
// ---------------------------------------------------------------------------
struct AttendArgs {
    const __nv_bfloat16 *Q;
    int Hq, H, G, PT;                      // PT = 128 / G positions of a query tile
    const int32_t *cu_q, *kv_lens;
    int total_q, max_q, max_kv_len;
    int pair0, n_tiles;
    const int32_t *order;
    const uint8_t *images;
    const TileMeta *meta;
    const float *ksigns, *vsigns;
    int n_splits, split_tiles;
    __nv_bfloat16 *out;
    float *lse;
    int x;                                 // blocks of 256 query rows of the longest run
    float *part_o, *part_ml;               // [split][pair][x][2 query tiles], see part_tile
    uint32_t *status;
};

// The run of sequence b: its first query, and how many are served.
__device__ __forceinline__ int run_of(const AttendArgs &a, int b, int *first, bool *cut) {
    const int q0 = a.cu_q[b], q1 = min(a.cu_q[b + 1], a.total_q);
    *first = q0;
    *cut = q0 >= 0 && q1 - q0 > a.max_q;
    return q0 >= 0 && q1 > q0 ? min(q1 - q0, a.max_q) : 0;
}

// The partial results of a query tile lie together: [row][2] (maximum, sum) and
// [D / 4][row][4], so that the threads of a warp, a row each, write side by side.
__device__ __forceinline__ int64_t part_tile(const AttendArgs &a, int split, int pl, int x, int tt) {
    return (((int64_t(split) * gridDim.y + pl) * a.x) + x) * 2 + tt;
}

// (m + log2 l) ln 2.  l may be 2^100 and m as far below zero (zero values), so
// l's exponent is taken to m before the rest, which is in [-1, 0), is added.
__device__ __forceinline__ float lse_of(float m, float l) {
    int e;
    const float f = frexpf(l, &e);
    return ((m + float(e)) + log2f(f)) * 0.6931471805599453f;
}

// Unnormalised Walsh-Hadamard transform of a vector in registers.
template <int D>
__device__ __forceinline__ void fwht_regs(float2 (&x)[D / 2]) {
#pragma unroll
    for (int i = 0; i < D / 2; ++i) x[i] = make_float2(x[i].x + x[i].y, x[i].x - x[i].y);
#pragma unroll
    for (int s = 1; s < D / 2; s <<= 1)
#pragma unroll
        for (int i = 0; i < D / 2; ++i)
            if ((i & s) == 0) {
                const float2 u = x[i], v = x[i + s];
                x[i] = add2(u, v);
                x[i + s] = fma2(v, make_float2(-1.f, -1.f), u);
            }
}
// x *= the signs of a rotation.
template <int D>
__device__ __forceinline__ void sign_regs(float2 (&x)[D / 2], const float *signs) {
#pragma unroll
    for (int i = 0; i < D / 4; ++i) {
        const float4 s = reinterpret_cast<const float4 *>(signs)[i];
        x[2 * i] = mul2(x[2 * i], make_float2(s.x, s.y));
        x[2 * i + 1] = mul2(x[2 * i + 1], make_float2(s.z, s.w));
    }
}

// The keys of value zero of a tile go to the sum alone: zs 2^zm in all, in units
// of 2^m.  They count as values of 2^-86 where that is above the reference, so
// that the sum stays below 2^127.  Returns m and l as they are then; has_o: there
// is an O to follow m.  Read from tensor memory again, before the loop's own 128
// registers of S are filled: asking for it costs every tile 1 % (8 runs of 1,024
// over up to 8,192 states, attention 408 -> 412 us), done on those registers 5 %.
template <int D>
__device__ __noinline__ float2 zero_keys(uint32_t ts, uint32_t to, const TileMeta *meta, float c2, float m, float l,
                                         bool has_o) {
    float zs = 0.f, zm = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        const uint32_t bits = meta->zero[c];
        if (bits == 0u) continue;
        float v[32], top = zm, part = 0.f;
        tc05::tmem_ld_32x32b_x32(ts + uint32_t(c * 32), reinterpret_cast<uint32_t(&)[32]>(v));
        tc05::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if ((bits >> e) & 1u) top = fmaxf(top, v[e]);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if ((bits >> e) & 1u) part += ex2_approx((v[e] - top) * c2);
        zs = fmaf(zs, ex2_approx((zm - top) * c2), part);
        zm = top;
    }
    zm *= c2;
    const bool up = zm - 86.f - m > 15.f;
    const float ref = up ? ceilf(zm) - 93.f : m, alpha = up ? exp2f(m - ref) : 1.f;
    l = fmaf(l, alpha, zs * exp2f(zm - ref));
    if (has_o && __any_sync(kFull, up)) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tc05::tmem_ld_32x32b_x32(to + uint32_t(c * 32), o);
            tc05::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc05::tmem_st_32x32b_x32(to + uint32_t(c * 32), o);
        }
        tc05::tmem_wait_st();
    }
    return make_float2(ref, l);
}

template <int D>
constexpr int ring_slots() { return D == 128 ? 5 : 8; }
constexpr int kMetaSlots = 8;
constexpr uint32_t kBarBytes = 512;
template <int D>
constexpr size_t attend_smem() {
    return (2 + ring_slots<D>()) * image_bytes(D) + kMetaSlots * sizeof(TileMeta) + kBarBytes + 1024;
}
// Three warpgroups: two of softmax rows, one with the MMA issuer's warp and
// the loader's.  The first two take registers that the third gives up
// (168 x 3 = 232 x 2 + 40): a row's 128 logits stay in registers.
constexpr int kAttendThreads = 384;
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 232;"); }
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 40;"); }

template <int D>
__global__ void __launch_bounds__(kAttendThreads, 1) cross_attend_kernel(const __grid_constant__ AttendArgs a) {
    constexpr uint32_t kImg = uint32_t(image_bytes(D));
    constexpr int NS = ring_slots<D>();
    constexpr uint32_t TO = 256;                          // TMEM columns: S / P of the tiles at 0 and 128, O behind
    wait_for_last();
    let_next_in();
    const int pl = a.order[blockIdx.y], pair = a.pair0 + pl, b = pair / a.H, h = pair - b * a.H, split = blockIdx.z;
    int q0;
    bool cut;
    const int nq = run_of(a, b, &q0, &cut);
    if (cut && blockIdx.x == 0 && h == 0 && split == 0 && threadIdx.x == 0) atomicOr(a.status, TQ_DEV_ROW);
    const int pos0 = int(blockIdx.x) * 2 * a.PT;
    if (pos0 >= nq) return;
    const int n_t = pos0 + a.PT < nq ? 2 : 1;
    const int len = min(max(a.kv_lens[b], 0), a.max_kv_len);
    const int tile0 = split * a.split_tiles;
    const int n = min((len + kTile - 1) / kTile - tile0, a.split_tiles);

    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
    const int tt = (tid >> 7) & 1, r = tid & 127;         // softmax threads: query tile and row
    const int qpos = pos0 + tt * a.PT + r / a.G;
    const bool row_ok = tid < 256 && r < a.PT * a.G && qpos < nq;
    const int64_t row = (int64_t(q0) + qpos) * a.Hq + h * a.G + r % a.G;
    const int64_t part = part_tile(a, split, pl, blockIdx.x, tt) * kTile;

    if (n <= 0) {                                         // no key of this split
        if (!row_ok) return;
        if (a.n_splits > 1) {
            *reinterpret_cast<float2 *>(a.part_ml + (part + r) * 2) = make_float2(-INFINITY, 0.f);
        } else {
            for (int i = 0; i < D / 8; ++i)
                reinterpret_cast<uint4 *>(a.out + row * D)[i] = make_uint4(0u, 0u, 0u, 0u);
            if (a.lse) a.lse[row] = -INFINITY;
        }
        return;
    }

    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_holder;
    __shared__ uint32_t abort_word;
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = sm, *ring = sm + 2 * kImg;
    TileMeta *smeta = reinterpret_cast<TileMeta *>(ring + NS * kImg);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smeta + kMetaSlots);
    uint64_t *kv_full = bars;                             // [NS] operand tile landed
    uint64_t *kv_empty = bars + 8;                        // [NS] its products done (commit)
    uint64_t *meta_full = bars + 16;                      // [8]
    uint64_t *s_full = bars + 24;                         // [2] S of a query tile done (commit)
    uint64_t *p_half = bars + 26;                         // [2] first 64 keys of P written, O rescaled (a lane of 4 warps)
    uint64_t *p_full = bars + 28;                         // [2] the rest
    uint64_t *o_done = bars + 30;                         // [2] last product of a tile done (commit)
    uint64_t *q_full = bars + 32;                         // queries staged (4 warps a tile)
    uint64_t *drained = bars + 33;                        // products in flight when a wait gave up
    volatile uint32_t *abort_flag = &abort_word;
    if (warp == 8) {
        tc05::tmem_alloc(&tmem_holder, 512);
        tc05::tmem_relinquish();
    }
    if (tid == 288) {
        for (int i = 0; i < NS; ++i) {
            tc05::mbar_init(&kv_full[i], 1);
            tc05::mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < kMetaSlots; ++i) tc05::mbar_init(&meta_full[i], 1);
        for (int i = 0; i < 2; ++i) {
            tc05::mbar_init(&s_full[i], 1);
            tc05::mbar_init(&p_half[i], 4);
            tc05::mbar_init(&p_full[i], 4);
            tc05::mbar_init(&o_done[i], 1);
        }
        tc05::mbar_init(q_full, uint32_t(4 * n_t));
        tc05::mbar_init(drained, 1);
        abort_word = 0u;
        tc05::fence_mbar_init();
    }
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = tmem_holder;
    bool timeout = false;

    if (warp >= 8) {
        fewer_registers();
    if (warp == 9) {
        // ================= loader: K(0), V(0), K(1), V(1), ... through one ring
        if (lane == 0) {
            const int64_t at = int64_t(pl) * a.n_tiles + tile0;
            const uint8_t *img = a.images + size_t(at) * 2 * kImg;
            int issued = 0;
            for (int i = 0; i < 2 * n; ++i) {
                const int s = i % NS, j = i >> 1;
                if (i >= NS && !wait_or_abort(&kv_empty[s], uint32_t(i / NS - 1) & 1u, abort_flag)) {
                    timeout = true;
                    break;
                }
                if ((i & 1) == 0) {
                    // the slot's last reader was tile j - 8, whose softmax is long done: the
                    // operand slot just found empty is of a later tile
                    tc05::mbar_expect_tx(&meta_full[j % kMetaSlots], uint32_t(sizeof(TileMeta)));
                    tc05::bulk_g2s(&smeta[j % kMetaSlots], a.meta + at + j, uint32_t(sizeof(TileMeta)),
                                   &meta_full[j % kMetaSlots]);
                }
                tc05::mbar_expect_tx(&kv_full[s], kImg);
                tc05::bulk_g2s(ring + s * kImg, img + size_t(i) * kImg, kImg, &kv_full[s]);
                issued = i + 1;
            }
            // copies in flight land before shared memory is given back
            for (int i = issued > NS ? issued - NS : 0; i < issued; ++i) {
                const int j = i >> 1;
                if (!wait_bounded(&kv_full[i % NS], uint32_t(i / NS) & 1u)) timeout = true;
                if ((i & 1) == 0 && !wait_bounded(&meta_full[j % kMetaSlots], uint32_t(j / kMetaSlots) & 1u))
                    timeout = true;
            }
        }
        __syncwarp();
    } else if (warp == 8) {
        // ================= MMA issuer: the whole warp walks the loop, so that
        // addresses and descriptors stay in uniform registers, and one lane
        // issues (a single lane's own loop took 70 to 115 cycles a product,
        // more than the 64 that it runs)
        constexpr uint32_t idesc_qk = tc05::idesc_f16_f32(128, 128);
        constexpr uint32_t idesc_pv = tc05::idesc_f16_f32(128, D) | tc05::kIdescBMajorMN;
        const bool lead = elect_one();
        const uint32_t tm = __shfl_sync(kFull, tmem, 0);
        const uint64_t dq = tc05::desc_kmajor_sw128(tc05::smem_u32(sQ));
        const uint64_t dk = tc05::desc_kmajor_sw128(tc05::smem_u32(ring));
        const uint64_t dv = tc05::desc_mnmajor_sw128(tc05::smem_u32(ring), 16384u, 1024u);
        auto wait_w = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(kFull, wait_or_abort(bar, parity, abort_flag));
        };
        auto qk = [&](int t, int slot) {                   // S_t = Q_t K^T, K in a ring slot
            const uint64_t A = dq + uint64_t(t) * (kImg >> 4), B = dk + uint64_t(slot) * (kImg >> 4);
            const uint32_t S = tm + uint32_t(t) * 128u;
            if (lead) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t o = (uint32_t(ks >> 2) * 16384u + uint32_t(ks & 3) * 32u) >> 4;
                    tc05::mma_f16(S, A + o, B + o, idesc_qk, ks > 0);
                }
                tc05::mma_commit(&s_full[t]);
            }
        };
        auto pv = [&](int t, int slot, int half, bool add) {   // O_t += P_t V over 64 keys, V in a ring slot
            const uint64_t B = dv + uint64_t(slot) * (kImg >> 4) + uint64_t(half) * (8192u >> 4);
            const uint32_t P = tm + uint32_t(t) * 128u + uint32_t(half) * 32u, O = tm + TO + uint32_t(t * D);
            if (lead) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    tc05::mma_f16_ts(O, P + uint32_t(ks) * 8u, B + uint32_t(ks) * (2048u >> 4), idesc_pv, add || ks > 0);
            }
        };
        auto release = [&](uint64_t *bar) {
            if (lead) tc05::mma_commit(bar);
        };
        int slot = 0;                                      // ring slot and phase of the next operand tile
        uint32_t phase = 0;
        auto next = [&](int *at) {                         // waits for it
            *at = slot;
            const bool ok = wait_w(&kv_full[slot], phase);
            if (++slot == NS) {
                slot = 0;
                phase ^= 1u;
            }
            return ok;
        };
        int k_slot = 0, v_slot = 0;
        bool started = false;
        bool ok = wait_w(q_full, 0u) && next(&k_slot);
        if (ok) {
            tc05::fence_after_sync();
            for (int t = 0; t < n_t; ++t) qk(t, k_slot);
            release(&kv_empty[k_slot]);
            started = true;
        }
        for (int j = 0; j < n && ok; ++j) {
            const bool more = j + 1 < n;
            ok = next(&v_slot) && (!more || next(&k_slot));
            for (int t = 0; t < n_t && ok; ++t) {
                const bool last = t == n_t - 1;
                ok = wait_w(&p_half[t], uint32_t(j) & 1u);
                if (!ok) break;
                tc05::fence_after_sync();
                pv(t, v_slot, 0, j > 0);
                ok = wait_w(&p_full[t], uint32_t(j) & 1u);
                if (!ok) break;
                tc05::fence_after_sync();
                pv(t, v_slot, 1, true);
                if (last) release(&kv_empty[v_slot]);
                if (more) {
                    // in issue order behind the product that reads P from the same columns
                    qk(t, k_slot);
                    if (last) release(&kv_empty[k_slot]);
                } else {
                    release(&o_done[t]);
                }
            }
        }
        timeout = !ok;
        if (timeout && started) {
            // what was issued completes before TMEM and shared memory are given back
            release(drained);
            wait_bounded(drained, 0u);
        }
        __syncwarp();
    }
    } else {
        more_registers();
    if (tt < n_t) {
        // ================= softmax: a thread per query row
        const uint32_t lrow = uint32_t((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lrow + uint32_t(tt) * 128u, to = tmem + lrow + TO + uint32_t(tt * D);
        float rowc = 1.f;
        bool finite = true;
        {
            float2 x[D / 2];
            if (row_ok) {
                const uint4 *src = reinterpret_cast<const uint4 *>(a.Q + row * D);
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 u = src[c];
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[4 * c + e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
                }
            } else {
#pragma unroll
                for (int i = 0; i < D / 2; ++i) x[i] = make_float2(0.f, 0.f);
            }
            sign_regs<D>(x, a.ksigns);
            fwht_regs<D>(x);
            float mx = 0.f;
            float2 bad = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < D / 2; ++i) {
                mx = fmaxf(mx, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
                bad = fma2(x[i], make_float2(0.f, 0.f), bad);
            }
            finite = bad.x + bad.y == 0.f;                 // a coordinate that is not finite spreads over the row
            int e;
            const float down = scale_to(finite ? mx : 0.f, 11, &e);
            // log2(e) / sqrt(d) of the logit, 1 / sqrt(d) of the rotation
            rowc = ldexpf(1.4426950408889634f / float(D), e);
            uint8_t *dst = sQ + uint32_t(tt) * kImg;
            const float2 down2 = make_float2(down, down);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 y = mul2(x[4 * c + k], down2);
                    w[k] = h2u(y.x, y.y);
                }
                *reinterpret_cast<uint4 *>(dst + (c >> 3) * 16384 + tc05::sw128_offset(uint32_t(r), uint32_t(c & 7))) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        tc05::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc05::mbar_arrive(q_full);
        // waits decided per warp, so the warp-wide TMEM accesses stay converged
        auto wait_w = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(kFull, wait_or_abort(bar, parity, abort_flag));
        };
        float m = -INFINITY, l = 0.f;                      // log2 units
        for (int j = 0; j < n; ++j) {
            if (!wait_w(&meta_full[j % kMetaSlots], uint32_t(j / kMetaSlots) & 1u)) {
                timeout = true;
                break;
            }
            const float4 sc = *reinterpret_cast<const float4 *>(&smeta[j % kMetaSlots]);
            if (!wait_w(&s_full[tt], uint32_t(j) & 1u)) {
                timeout = true;
                break;
            }
            tc05::fence_after_sync();
            const float c2 = fmaxf(rowc * sc.x, 1e-37f);
            if (__float_as_uint(sc.w) != 0u) {
                const float2 ml = zero_keys<D>(ts, to, smeta + j % kMetaSlots, c2, m, l, j > 0);
                m = ml.x;
                l = ml.y;
            }
            const uint4 mask = *reinterpret_cast<const uint4 *>(smeta[j % kMetaSlots].mask);
            float s[128];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                tc05::tmem_ld_32x32b_x32(ts + uint32_t(c * 32), reinterpret_cast<uint32_t(&)[32]>(s[c * 32]));
            tc05::tmem_wait_ld();
            if ((mask.x & mask.y & mask.z & mask.w) != 0xFFFFFFFFu) {
                const uint32_t mw[4] = {mask.x, mask.y, mask.z, mask.w};
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    if (!((mw[i >> 5] >> (i & 31)) & 1u)) s[i] = -INFINITY;
            }
            float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int i = 4; i < 124; i += 8)
#pragma unroll
                for (int u = 0; u < 4; ++u) mx4[u] = fmaxf(mx4[u], fmaxf(s[i + 2 * u], s[i + 2 * u + 1]));
#pragma unroll
            for (int u = 0; u < 4; ++u) mx4[u] = fmaxf(mx4[u], s[124 + u]);
            const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            const float top = fmaf(mx, c2, sc.y);
            // Set to 2^7 below the strongest weight, the reference moves only
            // when a tile's strongest leaves [2^-9, 2^15], so O is rescaled a
            // few times a row, not every tile.  It moves down, too: where one
            // strong key has a small value, the result is made of the others'
            // weights.  O and the sum, fp32, grow by 2^30 at most a time while
            // the sum is below 2^72: O, at most 2^16 times the sum, stays below 2^118.
            const float d = top - m;
            const bool move = d > 15.f || (d < -9.f && d > -1e30f && l < 0x1p72f);
            const float ref = fmaxf(ceilf(top) - 7.f, m - 30.f);   // whole numbers: factors are exact
            const float alpha = move ? exp2f(m - ref) : 1.f;
            if (move) {
                m = ref;
                l *= alpha;
            }
            if (j > 0 && __any_sync(kFull, move)) {
                // S of this tile was issued behind the last product into O: O is stable
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tc05::tmem_ld_32x32b_x32(to + uint32_t(c * 32), o);
                    tc05::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                    tc05::tmem_st_32x32b_x32(to + uint32_t(c * 32), o);
                }
            }
            const float off = m == -INFINITY ? 0.f : sc.y - m;
            const float2 c22 = make_float2(c2, c2), off2 = make_float2(off, off);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 x = fma2(make_float2(s[c * 32 + 2 * e], s[c * 32 + 2 * e + 1]), c22, off2);
                    const float2 w = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                    sum[e & 1] = add2(sum[e & 1], w);
                    p[e] = h2u(w.x, w.y);
                }
                tc05::tmem_st_32x32b_x16(ts + uint32_t(c * 16), p);
                if (c & 1) {
                    // 64 keys: their product may start.  One lane arrives for its
                    // warp: 128 arrivals on one barrier took some 400 cycles
                    tc05::tmem_wait_st();
                    tc05::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc05::mbar_arrive(c == 1 ? &p_half[tt] : &p_full[tt]);
                }
            }
            l = fmaf((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y), sc.z, l);
        }
        if (!timeout && !wait_w(&o_done[tt], 0u)) timeout = true;
        tc05::fence_after_sync();
        if (!finite) l = __uint_as_float(0x7FC00000u);
        uint32_t raw[D];
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            tc05::tmem_ld_32x32b_x32(to + uint32_t(c * 32), reinterpret_cast<uint32_t(&)[32]>(raw[c * 32]));
        tc05::tmem_wait_ld();
        float2 o[D / 2];
#pragma unroll
        for (int i = 0; i < D / 2; ++i) o[i] = make_float2(__uint_as_float(raw[2 * i]), __uint_as_float(raw[2 * i + 1]));
        if (row_ok && a.n_splits > 1) {
            float4 *dst = reinterpret_cast<float4 *>(a.part_o + part * D) + r;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) dst[i * kTile] = make_float4(o[2 * i].x, o[2 * i].y, o[2 * i + 1].x, o[2 * i + 1].y);
            *reinterpret_cast<float2 *>(a.part_ml + (part + r) * 2) = make_float2(m, l);
        } else if (row_ok) {
            fwht_regs<D>(o);
            const float inv = (l != l || l > 0.f ? 1.f / l : 0.f) * rsqrtf(float(D));
            sign_regs<D>(o, a.vsigns);
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + row * D);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(o[4 * c + e].x * inv, o[4 * c + e].y * inv);
                    w[e] = *reinterpret_cast<const uint32_t *>(&v);
                }
                dst[c] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (a.lse) a.lse[row] = l != l ? l : l > 0.f ? lse_of(m, l) : -INFINITY;
        }
    }
    }
    tc05::fence_before_sync();
    __syncthreads();
    if (warp == 8) {
        tc05::fence_after_sync();
        tc05::tmem_dealloc(tmem, 512);
    }
    if (timeout) atomicOr(a.status, TQ_DEV_WAIT_TIMEOUT);
}

// Merges the splits: eight threads a row (an eighth of its coordinates each),
// four rows a warp, so that a warp's loads are 64 bytes side by side, those of
// four splits on their way at once.
template <int D>
__global__ void __launch_bounds__(128) cross_merge_kernel(const __grid_constant__ AttendArgs a) {
    constexpr int Q = D / 8;                              // coordinates of a thread
    wait_for_last();
    const int lane = threadIdx.x & 31, eighth = lane >> 2;
    const int x = int(blockIdx.x) >> 4, tt = (int(blockIdx.x) >> 3) & 1;
    const int r = (int(blockIdx.x) & 7) * 16 + (threadIdx.x >> 5) * 4 + (lane & 3);
    const int pl = int(blockIdx.y), pair = a.pair0 + pl, b = pair / a.H, h = pair - b * a.H;
    int q0;
    bool cut;
    const int nq = run_of(a, b, &q0, &cut), qpos = (2 * x + tt) * a.PT + r / a.G;
    const bool ok = r < a.PT * a.G && qpos < nq;
    if (!__any_sync(kFull, ok)) return;
    const int64_t first = part_tile(a, 0, pl, x, tt) * kTile, step = part_tile(a, 1, pl, x, tt) * kTile - first;
    auto ml = [&](int s) {                                // a split without keys (or another run's row): sum 0
        return ok ? *reinterpret_cast<const float2 *>(a.part_ml + (first + s * step + r) * 2) : make_float2(-INFINITY, 0.f);
    };
    float M = -INFINITY;
#pragma unroll 8
    for (int s = 0; s < a.n_splits; ++s) {
        const float2 w = ml(s);
        if (w.y != 0.f) M = fmaxf(M, w.x);
    }
    float l = 0.f;
    float2 o[Q / 2];
#pragma unroll
    for (int i = 0; i < Q / 2; ++i) o[i] = make_float2(0.f, 0.f);
    for (int s0 = 0; s0 < a.n_splits; s0 += 4) {
        float f[4];
        float4 v[4][Q / 4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 w = s0 + k < a.n_splits ? ml(s0 + k) : make_float2(-INFINITY, 0.f);
            f[k] = w.y != 0.f ? exp2f(w.x - M) : 0.f;
            l = fmaf(w.y, f[k], l);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 *src = reinterpret_cast<const float4 *>(a.part_o + (first + (s0 + k) * step) * D) +
                                eighth * (Q / 4) * kTile + r;
#pragma unroll
            for (int i = 0; i < Q / 4; ++i) v[k][i] = f[k] != 0.f ? src[i * kTile] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < Q / 4; ++i) {
                o[2 * i] = fma2(make_float2(v[k][i].x, v[k][i].y), make_float2(f[k], f[k]), o[2 * i]);
                o[2 * i + 1] = fma2(make_float2(v[k][i].z, v[k][i].w), make_float2(f[k], f[k]), o[2 * i + 1]);
            }
    }
    // the transform's last three stages go across the row's threads
    fwht_regs<Q>(o);
#pragma unroll
    for (int bit = 4; bit <= 16; bit <<= 1) {
        const float sg = lane & bit ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < Q / 2; ++i) {
            const float2 y = make_float2(__shfl_xor_sync(kFull, o[i].x, bit), __shfl_xor_sync(kFull, o[i].y, bit));
            o[i] = fma2(o[i], make_float2(sg, sg), y);
        }
    }
    if (!ok) return;
    const int64_t row = (int64_t(q0) + qpos) * a.Hq + h * a.G + r % a.G;
    const float inv = (l != l || l > 0.f ? 1.f / l : 0.f) * rsqrtf(float(D));
    sign_regs<Q>(o, a.vsigns + eighth * Q);
    uint4 *dst = reinterpret_cast<uint4 *>(a.out + row * D + eighth * Q);
#pragma unroll
    for (int c = 0; c < Q / 8; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(o[4 * c + e].x * inv, o[4 * c + e].y * inv);
            w[e] = *reinterpret_cast<const uint32_t *>(&v);
        }
        dst[c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (a.lse && eighth == 0) a.lse[row] = l != l ? l : l > 0.f ? lse_of(M, l) : -INFINITY;
}

// Sizes of a call: the workspace holds the operand tiles of as many (sequence,
// KV head) pairs as fit kImageBudget (at least one), round after round.
constexpr size_t kImageBudget = size_t(1) << 30;

struct TcPlan {
    int n_tiles, pairs, round, x, n_splits, split_tiles;
    size_t off_order, off_meta, off_img, off_po, off_pml, total;
};

TcPlan tc_plan(const Layout &L, const CrossShape &s) {
    TcPlan p{};
    const int G = s.Hq / L.H, PT = kTile / G;
    p.n_tiles = (s.max_kv_len + kTile - 1) / kTile;
    if (p.n_tiles < 1) p.n_tiles = 1;
    p.pairs = s.B * L.H;
    const size_t pair_bytes = size_t(p.n_tiles) * 2 * image_bytes(L.d);
    size_t fit = kImageBudget / pair_bytes;
    if (fit < 1) fit = 1;
    if (fit > 65535) fit = 65535;
    p.round = int(fit < size_t(p.pairs) ? fit : size_t(p.pairs));
    p.x = (s.max_q + 2 * PT - 1) / (2 * PT);
    // The key axis is split where blocks are few: into pieces of four tiles or
    // more while the pieces fill the SMs but once, beyond that of eight or more
    // and up to two and a half blocks an SM (they run one after another, which
    // evens out runs and sequences of different lengths; every partial result
    // costs a write and a read).  Keys of 2 bits with a sketch, values of 4, 32
    // heads, against three waves of eight tiles everywhere: one run of 300 over
    // 1,500 states 41 us against 47, 8 of up to 77 over up to 4,096 94 against
    // 104, 2 of 512 over 4,096 125 against 158, but 2 of up to 77 over up to
    // 32,768 207 against 201.
    const int64_t blocks = int64_t(p.x) * p.round < 1 ? 1 : int64_t(p.x) * p.round;
    const int64_t once = 148 / blocks, more = 148 * 5 / 2 / blocks;
    int sp = int(once < p.n_tiles / 4 ? once : p.n_tiles / 4);
    const int sp8 = int(more < p.n_tiles / 8 ? more : p.n_tiles / 8);
    if (sp < sp8) sp = sp8;
    if (sp < 1) sp = 1;
    p.split_tiles = (p.n_tiles + sp - 1) / sp;
    p.n_splits = (p.n_tiles + p.split_tiles - 1) / p.split_tiles;
    size_t off = kWsHeader;
    auto take = [&](size_t bytes) { const size_t o = off; off += (bytes + 255) & ~size_t(255); return o; };
    p.off_order = take(size_t(p.round) * 4);
    p.off_meta = take(size_t(p.round) * p.n_tiles * sizeof(TileMeta));
    p.off_img = take(size_t(p.round) * pair_bytes);
    const size_t rows = size_t(p.round) * size_t(p.x) * 2 * kTile * p.n_splits;
    p.off_po = take(p.n_splits > 1 ? rows * L.d * 4 : 0);
    p.off_pml = take(p.n_splits > 1 ? rows * 8 : 0);
    p.total = off;
    return p;
}

template <int D>
int run_tc(const tq_params *kp, const tq_params *vp, const Layout &L, const void *Q, const CrossShape &s,
           const uint8_t *cache, int64_t num_blocks, void *out, float *lse, uint8_t *ws, cudaStream_t st) {
    const TcPlan p = tc_plan(L, s);
    // shared memory beyond the default is asked for once a device
    static std::atomic<uint64_t> asked{0};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
    if (!(asked.load(std::memory_order_acquire) & bit) || !bit) {
        e = cudaFuncSetAttribute(cross_expand_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(expand_smem<D>()));
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(cross_attend_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(attend_smem<D>()));
        if (e != cudaSuccess) return e;
        asked.fetch_or(bit, std::memory_order_release);
    }
    ExpandArgs x{};
    x.L = L;
    x.kp = kp->dev;
    x.vp = vp->dev;
    x.table = s.block_table;
    x.kv_lens = s.kv_lens;
    x.bt_stride = s.max_blocks;
    x.max_kv_len = s.max_kv_len;
    x.cache = cache;
    x.num_blocks = num_blocks;
    x.n_tiles = p.n_tiles;
    x.order = reinterpret_cast<int32_t *>(ws + p.off_order);
    x.B = s.B;
    x.images = ws + p.off_img;
    x.meta = reinterpret_cast<TileMeta *>(ws + p.off_meta);
    x.status = reinterpret_cast<uint32_t *>(ws);
    AttendArgs a{};
    a.Q = static_cast<const __nv_bfloat16 *>(Q);
    a.Hq = s.Hq;
    a.H = L.H;
    a.G = s.Hq / L.H;
    a.PT = kTile / a.G;
    a.cu_q = s.cu_q;
    a.kv_lens = s.kv_lens;
    a.total_q = s.total_q;
    a.max_q = s.max_q;
    a.max_kv_len = s.max_kv_len;
    a.n_tiles = p.n_tiles;
    a.order = x.order;
    a.images = x.images;
    a.meta = x.meta;
    a.ksigns = kp->dev.signs;
    a.vsigns = vp->dev.signs;
    a.x = p.x;
    a.n_splits = p.n_splits;
    a.split_tiles = p.split_tiles;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.part_o = reinterpret_cast<float *>(ws + p.off_po);
    a.part_ml = reinterpret_cast<float *>(ws + p.off_pml);
    a.status = x.status;
    for (int p0 = 0; p0 < p.pairs; p0 += p.round) {
        const int np = p.pairs - p0 < p.round ? p.pairs - p0 : p.round;
        x.pair0 = a.pair0 = p0;
        x.n_pairs = np;
        const int64_t items = int64_t(np) * p.n_tiles;
        cross_expand_kernel<D><<<unsigned(items < 296 ? items : 296), 256, expand_smem<D>(), st>>>(x);
        e = launch_next(cross_attend_kernel<D>, dim3(unsigned(p.x), unsigned(np), unsigned(p.n_splits)), kAttendThreads,
                        attend_smem<D>(), st, a);
        if (e == cudaSuccess && p.n_splits > 1)
            e = launch_next(cross_merge_kernel<D>, dim3(unsigned(p.x) * 16u, unsigned(np)), 128, 0, st, a);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

}  // namespace

// Expanding the states pays once and for all rows, decoding by rows pays for
// every one.  Where the tensor-core decode kernel serves the codec the two
// meet at about five queries a run (8 x 32 heads over 2,048 states: 75 against
// 80 us at four queries, 94 against 81 at six; 32 sequences: 195 against 244 at
// four, 289 against 247 at six); where the general one would, expanding is
// ahead from the first (8 x 1 query, d = 64: 191 against 46 us; FP8 keys in
// pages of 16: 246 against 80).
bool cross_tc_covers(const Layout &L, bool dense, const CrossShape &s) {
    if ((L.d != 64 && L.d != 128) || dense) return false;
    return s.max_q > 4 || dec128_resident(L, s.Hq / L.H) == 0;
}

size_t cross_tc_ws_bytes(const Layout &L, const CrossShape &s) { return tc_plan(L, s).total; }

int launch_cross_tc(const tq_params *kp, const tq_params *vp, const Layout &L, const void *Q, const CrossShape &s,
                    const uint8_t *cache, int64_t num_blocks, void *out, float *lse, uint8_t *ws, cudaStream_t st) {
    if (L.d == 128) return run_tc<128>(kp, vp, L, Q, s, cache, num_blocks, out, lse, ws, st);
    return run_tc<64>(kp, vp, L, Q, s, cache, num_blocks, out, lse, ws, st);
}

}  // namespace tq
