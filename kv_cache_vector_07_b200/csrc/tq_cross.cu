// Cross attention: runs of queries, each seeing the whole cache of its
// sequence (an encoder's states, of another length than the run).
//
//   l_t = (nhat_t <Rq, c[code_t]> + rho_t sqrt(pi/2)/m <S R q, 2 s_t - 1>) / sqrt(d)
//   o   = R_v^T sum_t softmax(l)_t nhat_v,t c_v[code_v,t]
//
// By rows: every query row becomes a decode row of its own, with its
// sequence's table row and length, and the decode kernels read the compressed
// pages once for each.  Right for every codec, rotation and head size; what it
// reads grows with the run, so it serves runs of a few queries and what the
// tensor-core way does not cover.  32 rows x 32 heads over up to 2,048 tokens of
// k3v4: 4 us for the rows, 10 to prepare the queries, 49 to read, 8 to join; the
// bytes alone are 7.
#include <cuda_runtime.h>

#include "tq_chain.cuh"
#include "tq_dev.cuh"

namespace tq {
namespace {

// One warp per query row of row0 .. row0 + n_rows - 1: its sequence (the last b with cu_q[b] <= row), that
// sequence's length and its table row.  Runs beside the queries' preparation,
// which it has nothing to do with (4 of 66 us for 32 rows, when it ran first).
__global__ void __launch_bounds__(128) cross_rows_kernel(CrossRows a) {
    let_next_in();
    const int lane = threadIdx.x & 31;
    const int at = int(blockIdx.x) * 4 + (threadIdx.x >> 5), row = a.row0 + at;
    if (at >= a.n_rows) return;
    int lo = 0, hi = a.B;                                  // cu_q[lo] <= row (or lo = 0), lo < hi
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_q[mid] <= row) lo = mid;
        else hi = mid;
    }
    int len = -1;
    const int begin = a.cu_q[lo];
    if (row >= begin && row < a.cu_q[lo + 1]) {
        if (row - begin < a.max_q) len = min(max(a.kv_lens[lo], 0), a.max_kv_len);
        else if (lane == 0) atomicOr(a.status, TQ_DEV_ROW);
    }
    if (lane == 0) a.row_len[at] = len;
    const int pages = len > 0 ? (len + a.P - 1) / a.P : 0;
    for (int j = lane; j < pages; j += 32)
        a.row_table[int64_t(at) * a.width + j] = a.table[int64_t(lo) * a.bt_stride + j];
    wait_for_last();         // what comes behind may read what the kernel before wrote
}

AttnShape rows_shape(const Layout &L, const CrossShape &s, int n) {
    AttnShape r{};
    r.n_seq = n;
    r.Hq = s.Hq;
    r.max_blocks = (s.max_kv_len + L.P - 1) / L.P;
    r.bt_stride = r.max_blocks;
    r.is_decode = 1;
    r.cross = 1;
    r.max_len = s.max_kv_len;
    return r;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// The queries are taken some at a time, so that what a round holds (prepared
// queries, one partial result a row, lengths, a table row for every query) stays
// within 128 MB whatever the number of queries, their heads and the states'
// length; a query alone takes what it needs.  65,536 rows of a head at most.  (A
// round of few rows has its keys split, which adds up to 2,400 x G partial results.)
struct RowsPlan {
    int n;                       // queries of a round
    size_t inner, lens, total;   // workspace of the decode kernels; the rows' lengths behind it; all
};
RowsPlan rows_plan(const Layout &L, const CrossShape &s) {
    RowsPlan p;
    const size_t width = size_t(rows_shape(L, s, 1).max_blocks);
    const size_t query = size_t(s.Hq) * (12 * size_t(L.d) + 8) + 4 * (width + 1);
    size_t most = (size_t(1) << 27) / query;
    if (most > size_t(65536 / s.Hq)) most = size_t(65536 / s.Hq);
    if (most < 1) most = 1;
    p.n = size_t(s.total_q) < most ? s.total_q : int(most);
    // the last round has fewer rows, which may be split where the others' are not
    const int rest = p.n ? s.total_q % p.n : 0;
    p.inner = up256(attn_ws_bytes(L, rows_shape(L, s, p.n)));
    if (rest) {
        const size_t last = up256(attn_ws_bytes(L, rows_shape(L, s, rest)));
        if (last > p.inner) p.inner = last;
    }
    p.lens = up256(4 * size_t(p.n));
    p.total = p.inner + p.lens + up256(4 * size_t(p.n) * width);
    return p;
}

}  // namespace

// The size does not know the rotation of the parameters: it covers both ways.
size_t cross_ws_bytes(const Layout &L, const CrossShape &s) {
    const size_t rows = rows_plan(L, s).total;
    if (!cross_tc_covers(L, false, s)) return rows;
    const size_t tc = cross_tc_ws_bytes(L, s);
    return tc > rows ? tc : rows;
}

int launch_cross_rows(const CrossRows &a, void *stream) {
    return launch_next(cross_rows_kernel, dim3(unsigned((a.n_rows + 3) / 4)), 128, 0, static_cast<cudaStream_t>(stream), a);
}

int launch_cross(const tq_params *kp, const tq_params *vp, const Layout &L, const void *Q, const CrossShape &s,
                 const uint8_t *cache, int64_t num_blocks, void *out, float *lse, uint8_t *ws, void *stream) {
    if (cross_tc_covers(L, kp->dev.rot || vp->dev.rot, s))
        return launch_cross_tc(kp, vp, L, Q, s, cache, num_blocks, out, lse, ws, static_cast<cudaStream_t>(stream));
    const RowsPlan p = rows_plan(L, s);
    const int n = p.n;
    AttnShape r = rows_shape(L, s, n);
    CrossRows a;
    a.cu_q = s.cu_q;
    a.table = s.block_table;
    a.kv_lens = s.kv_lens;
    a.B = s.B;
    a.max_q = s.max_q;
    a.bt_stride = s.max_blocks;
    a.max_kv_len = s.max_kv_len;
    a.P = L.P;
    a.width = r.max_blocks;
    a.row_len = reinterpret_cast<int32_t *>(ws + p.inner);
    a.row_table = reinterpret_cast<int32_t *>(ws + p.inner + p.lens);
    a.status = reinterpret_cast<uint32_t *>(ws);
    r.seq_lens = a.row_len;
    r.block_table = a.row_table;
    r.rows = &a;
    for (int q0 = 0; q0 < s.total_q; q0 += n) {
        a.row0 = q0;
        a.n_rows = r.n_seq = s.total_q - q0 < n ? s.total_q - q0 : n;
        const int64_t at = int64_t(q0) * s.Hq;
        const int e = launch_attention(kp, vp, L, static_cast<const uint16_t *>(Q) + at * L.d, r, cache, num_blocks,
                                       static_cast<uint16_t *>(out) + at * L.d, lse ? lse + at : nullptr, nullptr, 0, ws,
                                       p.inner, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace tq
