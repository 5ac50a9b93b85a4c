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
    a.heads_per_group = 4;
    a.n_groups = (heads + a.heads_per_group - 1) / a.heads_per_group;
    const int64_t blocks = (n * a.n_groups + 7) / 8;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == TQ_DTYPE_BF16) {
        if (rd.style == TQ_ROPE_HALF) run<__nv_bfloat16, TQ_ROPE_HALF>(a, unsigned(blocks), st);
        else run<__nv_bfloat16, TQ_ROPE_PAIRS>(a, unsigned(blocks), st);
    } else {
        if (rd.style == TQ_ROPE_HALF) run<float, TQ_ROPE_HALF>(a, unsigned(blocks), st);
        else run<float, TQ_ROPE_PAIRS>(a, unsigned(blocks), st);
    }
    return cudaGetLastError();
}

}  // namespace tq
