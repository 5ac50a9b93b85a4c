// RMS norm of every query and key head with the position rotation in the same
// pass: from slices of a QKV projection to the vectors that the write path
// and the attention calls take.
//
//   y = x / sqrt(mean(x^2) + eps) * w
//   pair (a, b) -> scale (a cos u - b sin u, b cos u + a sin u),
//   u = pos[axis(p)] * inv_freq[p]
//
// The pass reads and writes every head once and computes about ten operations
// a value, so memory bounds it for long inputs and the launch for short ones.
// Angles: pos * inv_freq in fp64 (31 + 24 bits; an fp32 product is off by up
// to 2^-24 of the angle, half a turn at a position of 5e7), turned into turns
// and reduced to [-1/2, 1/2] there; sin and cos are then taken in fp32 of the
// reduced angle.  They belong to the token, so a warp computes them once and
// uses them for all its heads.
#include <type_traits>

#include <cuda_runtime.h>

#include "tq_dev.cuh"

namespace tq {
namespace {

struct RopeArgs {
    tq_heads t[2];                // q, k (n_heads = 0: absent)
    const int32_t *pos;
    int64_t axis_stride;
    const float *inv_freq;
    int64_t n;
    int d, rot, n_groups, heads_per_group;
    float eps, scale;
    int w_f32;
    uint8_t axis[128];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

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
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// sin and cos of pos * f.
__device__ __forceinline__ void turn(int32_t pos, float f, float *s, float *c) {
    const double turns = double(pos) * double(f) * 0.15915494309189535;   // 1 / (2 pi)
    sincospif(2.f * float(turns - rint(turns)), s, c);
}

__device__ __forceinline__ float weight_at(const void *w, int i, int f32) {
    return f32 ? static_cast<const float *>(w)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[i]);
}

// One warp per (token, group of heads); lane l holds units l, l + 32, ... of
// a head, a unit being a rotated pair or two neighbouring coordinates that do
// not turn.  Any strides and any even d.
template <typename T, int STYLE, int U>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t task = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t tok = task / a.n_groups;
    const int group = int(task - tok * a.n_groups);
    if (tok >= a.n) return;
    const int pairs = a.rot / 2, units = a.d / 2;
    int i0[U], i1[U];
    float sn[U], cs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int p = lane + 32 * u;
        i0[u] = STYLE == TQ_ROPE_HALF && p < pairs ? p : 2 * p;
        i1[u] = STYLE == TQ_ROPE_HALF && p < pairs ? p + pairs : 2 * p + 1;
        sn[u] = 0.f;
        cs[u] = 1.f;
        if (p < pairs) {
            turn(a.pos[a.axis[p] * a.axis_stride + tok], a.inv_freq[p], &sn[u], &cs[u]);
            sn[u] *= a.scale;
            cs[u] *= a.scale;
        }
    }
    const int all = a.t[0].n_heads + a.t[1].n_heads;
    const int h1 = min(all, (group + 1) * a.heads_per_group);
    for (int hh = group * a.heads_per_group; hh < h1; ++hh) {
        const bool is_k = hh >= a.t[0].n_heads;
        const tq_heads &t = a.t[is_k];
        const int h = is_k ? hh - a.t[0].n_heads : hh;
        const T *x = static_cast<const T *>(t.x) + tok * t.tok_stride + h * t.head_stride;
        T *out = static_cast<T *>(t.out) + tok * t.out_tok_stride + h * t.out_head_stride;
        float v0[U], v1[U], ss = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = lane + 32 * u < units;
            v0[u] = in ? to_f(x[i0[u]]) : 0.f;
            v1[u] = in ? to_f(x[i1[u]]) : 0.f;
            ss = fmaf(v0[u], v0[u], fmaf(v1[u], v1[u], ss));
        }
        if (t.weight) {
            const float r = 1.f / sqrtf(warp_sum(ss) / float(a.d) + a.eps);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (lane + 32 * u < units) {
                    v0[u] *= r * weight_at(t.weight, i0[u], a.w_f32);
                    v1[u] *= r * weight_at(t.weight, i1[u], a.w_f32);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (lane + 32 * u < units) {
                const bool turns = lane + 32 * u < pairs;     // the rest is written as it is (an infinity stays one)
                put(out + i0[u], turns ? v0[u] * cs[u] - v1[u] * sn[u] : v0[u]);
                put(out + i1[u], turns ? v1[u] * cs[u] + v0[u] * sn[u] : v1[u]);
            }
    }
}

// A lane's two chunks of four coordinates as the firsts a and the seconds b of
// its four pairs, and back (rounded once).  HALVES: a and b are one chunk each;
// else (a, b) alternate.
__device__ __forceinline__ void to_f(const uint2 &c, float (&v)[4]) {
    v[0] = __uint_as_float(c.x << 16);
    v[1] = __uint_as_float(c.x & 0xFFFF0000u);
    v[2] = __uint_as_float(c.y << 16);
    v[3] = __uint_as_float(c.y & 0xFFFF0000u);
}
__device__ __forceinline__ void to_f(const uint4 &c, float (&v)[4]) {
    v[0] = __uint_as_float(c.x);
    v[1] = __uint_as_float(c.y);
    v[2] = __uint_as_float(c.z);
    v[3] = __uint_as_float(c.w);
}
__device__ __forceinline__ void from_f(uint2 &c, float v0, float v1, float v2, float v3) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v0, v1), b = __floats2bfloat162_rn(v2, v3);
    c = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}
__device__ __forceinline__ void from_f(uint4 &c, float v0, float v1, float v2, float v3) {
    c = make_uint4(__float_as_uint(v0), __float_as_uint(v1), __float_as_uint(v2), __float_as_uint(v3));
}
template <bool HALVES, typename C>
__device__ __forceinline__ void unpack(const C &c0, const C &c1, float2 (&a)[2], float2 (&b)[2]) {
    float x[4], y[4];
    to_f(c0, x);
    to_f(c1, y);
    a[0] = HALVES ? make_float2(x[0], x[1]) : make_float2(x[0], x[2]);
    a[1] = HALVES ? make_float2(x[2], x[3]) : make_float2(y[0], y[2]);
    b[0] = HALVES ? make_float2(y[0], y[1]) : make_float2(x[1], x[3]);
    b[1] = HALVES ? make_float2(y[2], y[3]) : make_float2(y[1], y[3]);
}
template <bool HALVES, typename C>
__device__ __forceinline__ void repack(C &c0, C &c1, const float2 (&a)[2], const float2 (&b)[2]) {
    if (HALVES) {
        from_f(c0, a[0].x, a[0].y, a[1].x, a[1].y);
        from_f(c1, b[0].x, b[0].y, b[1].x, b[1].y);
    } else {
        from_f(c0, a[0].x, b[0].x, a[0].y, b[0].y);
        from_f(c1, a[1].x, b[1].x, a[1].y, b[1].y);
    }
}

// sin and cos (times the scale) of a lane's four pairs: every lane computes PER
// of them, and takes the rest from the lanes of the other heads.
template <typename T, int LPH>
__device__ __forceinline__ void lane_angles(const RopeArgs &a, int64_t tok, int u, int sub, bool turns, float2 (&sn)[2],
                                            float2 (&cs)[2]) {
    constexpr int CE = 4, HPS = 32 / LPH, PER = CE / HPS > 1 ? CE / HPS : 1;
    float s1[PER], k1[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int p = u * CE + (sub * PER + i) % CE;
        s1[i] = 0.f;
        k1[i] = 1.f;
        if (turns) {
            const double r = double(a.pos[a.axis[p] * a.axis_stride + tok]) * double(a.inv_freq[p]) *
                             0.15915494309189535;   // turns
            const float f = float(r - rint(r));
            if (sizeof(T) == 2) {
                // |angle| <= pi: the fast functions are within 2^-20.9
                // there, 4,000 times finer than half a bf16 step
                __sincosf(f * 6.283185307179586f, &s1[i], &k1[i]);
            } else {
                sincospif(2.f * f, &s1[i], &k1[i]);
            }
            s1[i] *= a.scale;
            k1[i] *= a.scale;
        }
    }
#pragma unroll
    for (int i = 0; i < CE; ++i) {
        const int from = (i / PER) * LPH + u;
        const float s = __shfl_sync(kFull, s1[i % PER], from), c = __shfl_sync(kFull, k1[i % PER], from);
        if (i & 1) {
            sn[i / 2].y = s;
            cs[i / 2].y = c;
        } else {
            sn[i / 2].x = s;
            cs[i / 2].x = c;
        }
    }
}

// The same where everything is aligned to chunks of four coordinates (8 bytes
// of bf16, 16 of fp32): a lane holds two chunks of a head whose coordinates
// pair up (TQ_ROPE_HALF: chunk c of either half; TQ_ROPE_PAIRS, and what does
// not turn: neighbouring chunks), LPH = d / 8 lanes a head, 32 / LPH heads a
// step, two steps' loads in flight.
// 32,768 tokens x 40 heads of 128 bf16: 381 us by the kernel above (2-byte
// accesses, and its angles' arithmetic for four heads only); 146 us with
// 16-byte chunks (80 registers and spills: too few warps to cover the loads),
// 125 us (82 % of the measured copy rate) with these and 64 registers.
template <typename T, int STYLE, int LPH>
__global__ void __launch_bounds__(256, 4) rope_chunk_kernel(const __grid_constant__ RopeArgs a) {
    using Chunk = std::conditional_t<sizeof(T) == 2, uint2, uint4>;
    constexpr int CE = 4, HPS = 32 / LPH, N2 = 2;
    const int lane = threadIdx.x & 31, u = lane % LPH, sub = lane / LPH;
    const int64_t task = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t tok = task / a.n_groups;
    const int group = int(task - tok * a.n_groups);
    if (tok >= a.n) return;
    const int pairs = a.rot / 2;
    const bool turns = u * CE < pairs;                // the lane's pairs u CE .. u CE + CE - 1 turn
    const bool halves = STYLE == TQ_ROPE_HALF;        // a lane whose coordinates do not turn may split its chunks anyhow
    const int e0 = halves && turns ? u * CE : 2 * u * CE;
    const int e1 = halves && turns ? pairs + u * CE : (2 * u + 1) * CE;
    const int nq = a.t[0].n_heads, all = nq + a.t[1].n_heads;
    const int h0 = group * a.heads_per_group, h1 = min(all, h0 + a.heads_per_group);

    float2 sn[N2], cs[N2];
    bool angles = false;
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
        const int base = t ? nq : 0;
        const int lo = max(h0, base) - base, hi = min(h1, t ? all : nq) - base;
        if (lo >= hi) continue;                       // the same for the whole warp
        const tq_heads &T_ = a.t[t];
        const T *x = static_cast<const T *>(T_.x) + tok * T_.tok_stride + int64_t(lo + sub) * T_.head_stride;
        T *out = static_cast<T *>(T_.out) + tok * T_.out_tok_stride + int64_t(lo + sub) * T_.out_head_stride;
        const int64_t xs = HPS * T_.head_stride, os = HPS * T_.out_head_stride;
        Chunk c0[2], c1[2];                           // two steps ahead
        auto load = [&](int k, int g) {
            c0[k] = c1[k] = Chunk{};
            if (g < hi) {
                c0[k] = *reinterpret_cast<const Chunk *>(x + e0);
                c1[k] = *reinterpret_cast<const Chunk *>(x + e1);
            }
            x += xs;
        };
        load(0, lo + sub);
        load(1, lo + sub + HPS);
        Chunk w0{}, w1{};
        const bool norm = T_.weight != nullptr, same = a.w_f32 == (sizeof(T) == 4);
        if (norm && same) {
            w0 = *reinterpret_cast<const Chunk *>(static_cast<const T *>(T_.weight) + e0);
            w1 = *reinterpret_cast<const Chunk *>(static_cast<const T *>(T_.weight) + e1);
        }
        if (!angles) {
            // behind the first loads; every lane computes PER of its CE angles
            // and takes the rest from the lanes of the other heads
            angles = true;
            lane_angles<T, LPH>(a, tok, u, sub, turns, sn, cs);
        }
        for (int g0 = lo; g0 < hi; g0 += 2 * HPS) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int g = g0 + k * HPS + sub;
                float2 va[N2], vb[N2];
                unpack<STYLE == TQ_ROPE_HALF>(c0[k], c1[k], va, vb);
                load(k, g + 2 * HPS);
                if (norm) {
                    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < N2; ++i) ss = fma2(va[i], va[i], fma2(vb[i], vb[i], ss));
                    float sum = ss.x + ss.y;
#pragma unroll
                    for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
                    const float r = 1.f / sqrtf(sum / float(a.d) + a.eps);
                    float2 wa[N2], wb[N2];
                    if (same) {
                        unpack<STYLE == TQ_ROPE_HALF>(w0, w1, wa, wb);
                    } else {
#pragma unroll
                        for (int i = 0; i < N2; ++i) {
                            const int f0 = halves ? e0 + 2 * i : e0 + 4 * i, step = halves ? 1 : 2;
                            const int s0 = halves ? e1 + 2 * i : e0 + 4 * i + 1;
                            wa[i] = make_float2(weight_at(T_.weight, f0, a.w_f32), weight_at(T_.weight, f0 + step, a.w_f32));
                            wb[i] = make_float2(weight_at(T_.weight, s0, a.w_f32), weight_at(T_.weight, s0 + step, a.w_f32));
                        }
                    }
                    const float2 r2 = make_float2(r, r);
#pragma unroll
                    for (int i = 0; i < N2; ++i) {
                        va[i] = mul2(va[i], mul2(r2, wa[i]));
                        vb[i] = mul2(vb[i], mul2(r2, wb[i]));
                    }
                }
                if (turns) {
#pragma unroll
                    for (int i = 0; i < N2; ++i) {
                        const float2 p = va[i], q = vb[i], ns = make_float2(-sn[i].x, -sn[i].y);
                        va[i] = fma2(p, cs[i], mul2(q, ns));
                        vb[i] = fma2(q, cs[i], mul2(p, sn[i]));
                    }
                }
                Chunk o0, o1;
                repack<STYLE == TQ_ROPE_HALF>(o0, o1, va, vb);
                if (g < hi) {
                    *reinterpret_cast<Chunk *>(out + e0) = o0;
                    *reinterpret_cast<Chunk *>(out + e1) = o1;
                }
                out += os;
            }
        }
    }
}

// The same for tokens of few heads (two steps' worth, q and k together): all of
// a token's loads are on their way at once, where the kernel above waits for q
// and for k in turn, which is all that it does there (52,424 tokens x 3 heads of
// 64 fp32: 27 us against 72; 18,444 x 5 of 64 bf16: 12 against 16).
template <typename T, int STYLE, int LPH>
__global__ void __launch_bounds__(256) rope_few_kernel(const __grid_constant__ RopeArgs a) {
    using Chunk = std::conditional_t<sizeof(T) == 2, uint2, uint4>;
    constexpr int CE = 4, HPS = 32 / LPH;
    constexpr bool halves = STYLE == TQ_ROPE_HALF;
    const int lane = threadIdx.x & 31, u = lane % LPH, sub = lane / LPH;
    const int64_t tok = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (tok >= a.n) return;
    const int pairs = a.rot / 2;
    const bool turns = u * CE < pairs;
    const int e0 = halves && turns ? u * CE : 2 * u * CE;
    const int e1 = halves && turns ? pairs + u * CE : (2 * u + 1) * CE;
    const int nq = a.t[0].n_heads, all = nq + a.t[1].n_heads;
    const bool same = a.w_f32 == (sizeof(T) == 4);
    Chunk c0[2], c1[2], w0[2], w1[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int g = k * HPS + sub;
        const tq_heads &t = a.t[g >= nq];
        c0[k] = c1[k] = w0[k] = w1[k] = Chunk{};
        if (g < all) {
            const T *x = static_cast<const T *>(t.x) + tok * t.tok_stride + int64_t(g >= nq ? g - nq : g) * t.head_stride;
            c0[k] = *reinterpret_cast<const Chunk *>(x + e0);
            c1[k] = *reinterpret_cast<const Chunk *>(x + e1);
            if (t.weight && same) {
                w0[k] = *reinterpret_cast<const Chunk *>(static_cast<const T *>(t.weight) + e0);
                w1[k] = *reinterpret_cast<const Chunk *>(static_cast<const T *>(t.weight) + e1);
            }
        }
    }
    float2 sn[2], cs[2];
    lane_angles<T, LPH>(a, tok, u, sub, turns, sn, cs);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int g = k * HPS + sub;
        const tq_heads &t = a.t[g >= nq];
        float2 va[2], vb[2];
        unpack<halves>(c0[k], c1[k], va, vb);
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 2; ++i) ss = fma2(va[i], va[i], fma2(vb[i], vb[i], ss));
        float sum = ss.x + ss.y;
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        if (g >= all) continue;                       // behind the last shuffle of this step
        if (t.weight) {
            const float r = 1.f / sqrtf(sum / float(a.d) + a.eps);
            float2 wa[2], wb[2];
            if (same) {
                unpack<halves>(w0[k], w1[k], wa, wb);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int f0 = halves ? e0 + 2 * i : e0 + 4 * i, step = halves ? 1 : 2;
                    const int s0 = halves ? e1 + 2 * i : e0 + 4 * i + 1;
                    wa[i] = make_float2(weight_at(t.weight, f0, a.w_f32), weight_at(t.weight, f0 + step, a.w_f32));
                    wb[i] = make_float2(weight_at(t.weight, s0, a.w_f32), weight_at(t.weight, s0 + step, a.w_f32));
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                va[i] = mul2(va[i], mul2(make_float2(r, r), wa[i]));
                vb[i] = mul2(vb[i], mul2(make_float2(r, r), wb[i]));
            }
        }
        if (turns) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 p = va[i], q = vb[i], ns = make_float2(-sn[i].x, -sn[i].y);
                va[i] = fma2(p, cs[i], mul2(q, ns));
                vb[i] = fma2(q, cs[i], mul2(p, sn[i]));
            }
        }
        T *out = static_cast<T *>(t.out) + tok * t.out_tok_stride + int64_t(g >= nq ? g - nq : g) * t.out_head_stride;
        Chunk o0, o1;
        repack<halves>(o0, o1, va, vb);
        *reinterpret_cast<Chunk *>(out + e0) = o0;
        *reinterpret_cast<Chunk *>(out + e1) = o1;
    }
}

template <typename T, int STYLE, int LPH>
void run_chunk_lanes(const RopeArgs &a, unsigned blocks, unsigned threads, cudaStream_t st) {
    if (a.t[0].n_heads + a.t[1].n_heads <= 2 * (32 / LPH)) rope_few_kernel<T, STYLE, LPH><<<blocks, threads, 0, st>>>(a);
    else rope_chunk_kernel<T, STYLE, LPH><<<blocks, threads, 0, st>>>(a);
}

template <typename T, int STYLE>
bool run_chunk(const RopeArgs &a, unsigned blocks, unsigned threads, cudaStream_t st) {
    switch (a.d / 8) {
        case 1: run_chunk_lanes<T, STYLE, 1>(a, blocks, threads, st); return true;
        case 2: run_chunk_lanes<T, STYLE, 2>(a, blocks, threads, st); return true;
        case 4: run_chunk_lanes<T, STYLE, 4>(a, blocks, threads, st); return true;
        case 8: run_chunk_lanes<T, STYLE, 8>(a, blocks, threads, st); return true;
        case 16: run_chunk_lanes<T, STYLE, 16>(a, blocks, threads, st); return true;
        case 32: run_chunk_lanes<T, STYLE, 32>(a, blocks, threads, st); return true;
    }
    return false;
}

// Whether every vector and weight lies on a chunk boundary and d is a power of
// two (LPH lanes a head divide the warp).
bool chunks_fit(const RopeArgs &a, int es) {
    if ((a.d & (a.d - 1)) || a.d < 8 || a.rot % 8) return false;
    const int bytes = 4 * es;
    for (const tq_heads &t : a.t) {
        if (!t.n_heads) continue;
        if ((t.tok_stride | t.head_stride | t.out_tok_stride | t.out_head_stride) % 4) return false;
        if ((reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.out)) % bytes) return false;
        if (reinterpret_cast<uintptr_t>(t.weight) % (a.w_f32 ? 16 : 8)) return false;
    }
    return true;
}

template <typename T, int STYLE>
void run(const RopeArgs &a, unsigned blocks, cudaStream_t st) {
    if (a.d <= 64) rope_kernel<T, STYLE, 1><<<blocks, 256, 0, st>>>(a);
    else if (a.d <= 128) rope_kernel<T, STYLE, 2><<<blocks, 256, 0, st>>>(a);
    else rope_kernel<T, STYLE, 4><<<blocks, 256, 0, st>>>(a);
}

}  // namespace

int launch_rope(const tq_rope_desc &rd, int dtype, int w_dtype, int64_t n, const tq_heads *q, const tq_heads *k,
                const int32_t *positions, int64_t axis_stride, const float *inv_freq, void *stream) {
    RopeArgs a{};
    if (q) a.t[0] = *q;
    if (k) a.t[1] = *k;
    a.pos = positions;
    a.axis_stride = axis_stride;
    a.inv_freq = inv_freq;
    a.n = n;
    a.d = rd.d;
    a.rot = rd.rot_dim;
    a.eps = rd.eps;
    a.scale = rd.scale;
    a.w_f32 = w_dtype == TQ_DTYPE_F32;
    for (int p = 0; p < rd.rot_dim / 2; ++p) a.axis[p] = rd.pair_axis[p];
    const int heads = a.t[0].n_heads + a.t[1].n_heads;
    const int es = dtype == TQ_DTYPE_BF16 ? 2 : 4;
    const bool chunks = chunks_fit(a, es);
    // heads of a warp: all of a token's where there are tokens enough to fill
    // the GPU (its angles are then computed once), few where there are not
    const int step = chunks ? 2 * (256 / a.d) : 4;
    const int64_t want = int64_t(148) * 32;            // warps
    int64_t per = chunks ? n * heads / want / step * step : 4;
    if (per < step) per = step;
    if (per > heads) per = (heads + step - 1) / step * step;
    a.heads_per_group = int(per);
    a.n_groups = (heads + a.heads_per_group - 1) / a.heads_per_group;
    const int64_t tasks = n * a.n_groups;
    const unsigned threads = chunks && tasks < 8 * 148 ? 64u : 256u;
    const int64_t blocks = (tasks + threads / 32 - 1) / (threads / 32);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (chunks) {
        if (dtype == TQ_DTYPE_BF16) {
            if (rd.style == TQ_ROPE_HALF) run_chunk<__nv_bfloat16, TQ_ROPE_HALF>(a, unsigned(blocks), threads, st);
            else run_chunk<__nv_bfloat16, TQ_ROPE_PAIRS>(a, unsigned(blocks), threads, st);
        } else {
            if (rd.style == TQ_ROPE_HALF) run_chunk<float, TQ_ROPE_HALF>(a, unsigned(blocks), threads, st);
            else run_chunk<float, TQ_ROPE_PAIRS>(a, unsigned(blocks), threads, st);
        }
    } else if (dtype == TQ_DTYPE_BF16) {
        if (rd.style == TQ_ROPE_HALF) run<__nv_bfloat16, TQ_ROPE_HALF>(a, unsigned(blocks), st);
        else run<__nv_bfloat16, TQ_ROPE_PAIRS>(a, unsigned(blocks), st);
    } else {
        if (rd.style == TQ_ROPE_HALF) run<float, TQ_ROPE_HALF>(a, unsigned(blocks), st);
        else run<float, TQ_ROPE_PAIRS>(a, unsigned(blocks), st);
    }
    return cudaGetLastError();
}

}  // namespace tq
