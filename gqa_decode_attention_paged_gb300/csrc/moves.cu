// Moving cached rows when one of several candidates is taken: the accepted
// path of a tree of drafted tokens to the front of its nodes, and the block
// that each beam of a search writes next.
//
// Both copy stored bytes as they are (16-byte pieces; a 4-bit value row's
// (scale, zero point) pair is 8), whatever the pool's type.  What bounds them
// is latency: a few rows of 4 KiB per sequence move, behind a chain of
// dependent reads (lengths and choices, then table entries, then rows).  So
// every thread block handles one (sequence or beam, KV head), all of a step's
// reads are issued at once, and nothing is staged.  In a graph, 8 KV heads of
// 128: 64 sequences that keep up to 7 of 26 nodes take 2.4 us, 200 on 4-bit rows
// 2.8 us; 16 new beams 2.3 us, 640 with tables of 128 blocks 5.3 us (13.6 MB: 2.6
// TB/s).
#include <algorithm>

#include "pkv_internal.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;

struct CommitArgs {
    uint8_t *pool;
    int64_t num_blocks;
    int n_kv;
    const int32_t *qo_indptr;     // [batch + 1]
    const int32_t *accepted;      // [batch][most]
    int most;
    const int32_t *count;         // [batch]
    const int32_t *block_tables;
    int W;
    const int32_t *context_lens;  // [batch], the nodes included
    int32_t *new_lens;            // [batch]
    unsigned *err;
};

// One (sequence, KV head).  Row accepted[i] goes to place i; as accepted is
// ascending (accepted[i] >= i), a step of rows i0 .. i0 + n - 1 writes no place
// that a later step reads, and within a step all rows are read before any is
// written.
template <int D, int KV>
__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const __grid_constant__ CommitArgs a)
{
    constexpr int ROWB = (int)kv_row_bytes(KV, D);
    constexpr int64_t ENTRY = kv_entry_bytes(KV, D);
    constexpr int PIECES = ROWB / 16;            // of a key (or value) row
    constexpr int RPS = kThreads / (2 * PIECES); // rows that a step's threads take at once
    constexpr int U = 4;                         // such groups of rows in a step
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.x, g = blockIdx.y, tid = threadIdx.x;
    const int32_t lo = a.qo_indptr[b], hi = a.qo_indptr[b + 1], n = a.count[b];
    const int32_t cap = a.W * kBlockSize, C = a.context_lens[b];
    const int32_t *acc = a.accepted + (int64_t)b * a.most;
    // (64 bits: an indptr may hold any numbers)
    const int64_t T = (int64_t)hi - lo;
    const int32_t first = (int32_t)max((int64_t)0, min((int64_t)max(C, 0), (int64_t)cap) - max(T, (int64_t)0));
    bool bad = lo < 0 || T < 0 || C < T || C > cap || n < 0 || n > a.most || n > T;
    if (!bad)
        for (int i = tid; i < n; i += kThreads) bad |= acc[i] >= T || acc[i] <= (i > 0 ? acc[i - 1] : -1);
    bad = __syncthreads_or(bad);
    if (g == 0 && tid == 0) {
        a.new_lens[b] = bad ? first : first + n;
        if (bad) atomicOr(a.err, PKV_DEVERR_CTX_RANGE);
    }
    if (bad) return;
    const int32_t *trow = a.block_tables + (int64_t)b * a.W;
    // the entry of the KV head that holds a position, and the row in it; -1: no block of the pool
    auto find = [&](int pos, int &row) -> int64_t {
        const int32_t blk = trow[pos / kBlockSize];
        row = pos % kBlockSize;
        return blk >= 0 && blk < a.num_blocks ? (int64_t)blk * a.n_kv + g : -1;
    };
    const int sub = tid / (2 * PIECES), piece = tid % (2 * PIECES);
    const int off = (piece / PIECES) * kBlockSize * ROWB + (piece % PIECES) * 16;
    for (int i0 = 0; i0 < n; i0 += U * RPS) {
        uint4 x[U];
        [[maybe_unused]] float2 par[U];
        uint8_t *dst[U];
        [[maybe_unused]] uint8_t *pdst[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * RPS + sub;
            dst[u] = nullptr;
            if (i >= n) continue;
            const int from = acc[i];
            if (from == i) continue;
            int rs, rd;
            const int64_t es = find(first + from, rs), ed = find(first + i, rd);
            if (es < 0 || ed < 0) {
                if (piece == 0 && g == 0) atomicOr(a.err, PKV_DEVERR_BLOCK_RANGE);
                continue;
            }
            dst[u] = a.pool + ed * ENTRY + rd * ROWB + off;
            x[u] = *reinterpret_cast<const uint4 *>(a.pool + es * ENTRY + rs * ROWB + off);
            if constexpr (KV == PKV_INT4) {
                pdst[u] = a.pool + ed * ENTRY + i4_params_offset(D) + 8 * rd;
                if (piece == 0) par[u] = *reinterpret_cast<const float2 *>(a.pool + es * ENTRY + i4_params_offset(D) + 8 * rs);
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!dst[u]) continue;
            *reinterpret_cast<uint4 *>(dst[u]) = x[u];
            if constexpr (KV == PKV_INT4)
                if (piece == 0) *reinterpret_cast<float2 *>(pdst[u]) = par[u];
        }
    }
}

struct ReorderArgs {
    uint8_t *pool;
    int64_t num_blocks;
    int n_kv;
    const int32_t *parents;   // [batch * k]
    int beams, k;
    const int32_t *tables;    // [batch * beams][W]
    int W;
    const int32_t *lens;      // [batch * beams]
    const int32_t *spare;     // [batch * k]
    int32_t *tables_out;      // [batch * k][W]
    int32_t *lens_out;        // [batch * k]
    unsigned *err;
};

// One new beam and KV head (the first head's block writes the table row).  The
// beam's entries before the block that it writes next are its
// parent's; that block is the parent's for the parent's first child, and for
// every other child a spare one into which the filled rows are copied.
template <int D, int KV>
__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const __grid_constant__ ReorderArgs a)
{
    constexpr int ROWB = (int)kv_row_bytes(KV, D);
    constexpr int64_t ENTRY = kv_entry_bytes(KV, D);
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x, item = row / a.k;
    const int j = (int)(row - item * a.k);
    const int32_t *parents = a.parents + item * a.k;
    int p = parents[j];
    bool earlier = false;
    for (int i = tid; i < j; i += kThreads) earlier |= parents[i] == p;
    const bool other = __syncthreads_or(earlier);
    const bool lead = blockIdx.y == 0;
    if (p < 0 || p >= a.beams) {
        if (lead && tid == 0 && p != -1) atomicOr(a.err, PKV_DEVERR_BLOCK_RANGE);
        p = -1;
    }
    int L = 0;
    const int32_t *src_row = nullptr;
    if (p >= 0) {
        src_row = a.tables + (item * a.beams + p) * a.W;
        L = a.lens[item * a.beams + p];
        if (L < 0 || L > a.W * kBlockSize) {
            if (lead && tid == 0) atomicOr(a.err, PKV_DEVERR_CTX_RANGE);
            L = min(max(L, 0), a.W * kBlockSize);
        }
    }
    const int here = p >= 0 ? L / kBlockSize : -1, rows = L % kBlockSize;
    const int32_t fresh = a.spare[row];
    if (lead) {
        int32_t *out = a.tables_out + row * a.W;
        for (int e = tid; e < a.W; e += kThreads) {
            int32_t id = e <= here ? src_row[e] : -1;
            if (e == here && other) id = fresh;
            out[e] = id;
        }
        if (tid == 0) a.lens_out[row] = L;
    }
    if (p < 0 || !other || here >= a.W) return;
    const int32_t from = rows ? src_row[here] : 0;
    if (fresh < 0 || fresh >= a.num_blocks || from < 0 || from >= a.num_blocks) {
        if (lead && tid == 0) atomicOr(a.err, PKV_DEVERR_BLOCK_RANGE);
        return;
    }
    // the head's filled rows: `pieces` 16-byte pieces of keys, as many of values (and the rows' parameters)
    const int pieces = rows * ROWB / 16;
    const uint8_t *src = a.pool + ((int64_t)from * a.n_kv + blockIdx.y) * ENTRY;
    uint8_t *dst = a.pool + ((int64_t)fresh * a.n_kv + blockIdx.y) * ENTRY;
    constexpr int U = (2 * kBlockSize * ROWB / 16 + kThreads - 1) / kThreads;
    uint4 x[U];
    int at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = u * kThreads + tid;
        at[u] = i < 2 * pieces ? (i >= pieces ? kBlockSize * ROWB + (i - pieces) * 16 : i * 16) : -1;
        if (at[u] >= 0) x[u] = ldg_nc_v4(src + at[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (at[u] >= 0) *reinterpret_cast<uint4 *>(dst + at[u]) = x[u];
    if constexpr (KV == PKV_INT4) {
        if (tid < rows) {
            const int p_at = i4_params_offset(D) + 8 * tid;
            *reinterpret_cast<float2 *>(dst + p_at) = __ldg(reinterpret_cast<const float2 *>(src + p_at));
        }
    }
}

// kern<D, KV> for the pool's head size and type.
#define PKV_LAUNCH_BY_POOL(kern, grid, s, a)                                                             \
    (pool->d_head == 128                                                                                \
         ? (pool->dtype == PKV_BF16       ? launch_pdl(kern<128, PKV_BF16>, grid, dim3(kThreads), 0, s, a)     \
            : pool->dtype == PKV_FP8_E4M3 ? launch_pdl(kern<128, PKV_FP8_E4M3>, grid, dim3(kThreads), 0, s, a) \
                                          : launch_pdl(kern<128, PKV_INT4>, grid, dim3(kThreads), 0, s, a))    \
         : (pool->dtype == PKV_BF16       ? launch_pdl(kern<64, PKV_BF16>, grid, dim3(kThreads), 0, s, a)      \
            : pool->dtype == PKV_FP8_E4M3 ? launch_pdl(kern<64, PKV_FP8_E4M3>, grid, dim3(kThreads), 0, s, a)  \
                                          : launch_pdl(kern<64, PKV_INT4>, grid, dim3(kThreads), 0, s, a)))

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status paged_tree_commit(pkv_pool *pool, const int32_t *qo_indptr, const int32_t *accepted,
                                        int32_t max_accepted, const int32_t *n_accepted, const int32_t *block_tables,
                                        int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t batch,
                                        int32_t *new_lens, void *stream)
{
    const char *who = "paged_tree_commit";
    if (!pool) return fail(PKV_EINVAL, "%s: NULL pool", who);
    if (batch < 0 || batch > kMaxBatch) return fail(PKV_EINVAL, "%s: batch %d out of range", who, batch);
    if (max_accepted < 0) return fail(PKV_EINVAL, "%s: max_accepted < 0", who);
    if (max_blocks_per_seq <= 0 || max_blocks_per_seq > (1 << 24))
        return fail(PKV_EINVAL, "%s: max_blocks_per_seq %d out of range", who, max_blocks_per_seq);
    if (batch == 0) return PKV_OK;
    if (!qo_indptr || (!accepted && max_accepted) || !n_accepted || !block_tables || !context_lens || !new_lens)
        return fail(PKV_EINVAL, "%s: NULL device pointer", who);
    if (((uintptr_t)qo_indptr | (uintptr_t)accepted | (uintptr_t)n_accepted | (uintptr_t)block_tables |
         (uintptr_t)context_lens | (uintptr_t)new_lens) & 3u)
        return fail(PKV_EINVAL, "%s: arrays must be 4-byte aligned", who);
    const size_t n = (size_t)batch * 4;
    if (overlap(new_lens, n, context_lens, n) || overlap(new_lens, n, n_accepted, n) ||
        overlap(new_lens, n, qo_indptr, n + 4) || overlap(new_lens, n, accepted, n * max_accepted) ||
        overlap(new_lens, n, block_tables, n * max_blocks_per_seq))
        return fail(PKV_EINVAL, "%s: new_lens overlaps an input", who);
    pkv_status st = check_pool_device(pool, who);
    if (st != PKV_OK) return st;
    CommitArgs a;
    a.pool = static_cast<uint8_t *>(pool->k);
    a.num_blocks = pool->num_blocks;
    a.n_kv = pool->n_kv;
    a.qo_indptr = qo_indptr;
    a.accepted = accepted;
    a.most = max_accepted;
    a.count = n_accepted;
    a.block_tables = block_tables;
    a.W = max_blocks_per_seq;
    a.context_lens = context_lens;
    a.new_lens = new_lens;
    a.err = pool->err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)batch, (unsigned)pool->n_kv);
    LaunchScope ls(pool, kBlocks, s);
    cudaError_t e = PKV_LAUNCH_BY_POOL(tree_commit_kernel, grid, s, a);
    ls.done();
    if (e != cudaSuccess) return cuda_fail(e, "paged_tree_commit launch");
    return PKV_OK;
}

extern "C" pkv_status paged_beam_reorder(pkv_pool *pool, const int32_t *parents, int32_t batch, int32_t beams, int32_t k,
                                         const int32_t *block_tables, int32_t max_blocks_per_seq,
                                         const int32_t *context_lens, const int32_t *spare_blocks, int32_t *tables_out,
                                         int32_t *lens_out, void *stream)
{
    const char *who = "paged_beam_reorder";
    if (!pool) return fail(PKV_EINVAL, "%s: NULL pool", who);
    if (batch < 0 || beams <= 0 || k <= 0) return fail(PKV_EINVAL, "%s: batch < 0, or no beams", who);
    if (max_blocks_per_seq <= 0 || max_blocks_per_seq > (1 << 24))
        return fail(PKV_EINVAL, "%s: max_blocks_per_seq %d out of range", who, max_blocks_per_seq);
    if ((int64_t)batch * std::max(beams, k) > (1 << 24)) return fail(PKV_EUNSUPPORTED, "%s: more than 2^24 beams", who);
    if (batch == 0) return PKV_OK;
    if (!parents || !block_tables || !context_lens || !spare_blocks || !tables_out || !lens_out)
        return fail(PKV_EINVAL, "%s: NULL device pointer", who);
    if (((uintptr_t)parents | (uintptr_t)block_tables | (uintptr_t)context_lens | (uintptr_t)spare_blocks |
         (uintptr_t)tables_out | (uintptr_t)lens_out) & 3u)
        return fail(PKV_EINVAL, "%s: arrays must be 4-byte aligned", who);
    const size_t nin = (size_t)batch * beams * 4, nout = (size_t)batch * k * 4, W = (size_t)max_blocks_per_seq;
    const void *outs[2] = {tables_out, lens_out};
    const size_t sizes[2] = {nout * W, nout};
    for (int i = 0; i < 2; ++i)
        if (overlap(outs[i], sizes[i], parents, nout) || overlap(outs[i], sizes[i], block_tables, nin * W) ||
            overlap(outs[i], sizes[i], context_lens, nin) || overlap(outs[i], sizes[i], spare_blocks, nout))
            return fail(PKV_EINVAL, "%s: an output overlaps an input", who);
    if (overlap(tables_out, nout * W, lens_out, nout)) return fail(PKV_EINVAL, "%s: the outputs overlap", who);
    pkv_status st = check_pool_device(pool, who);
    if (st != PKV_OK) return st;
    ReorderArgs a;
    a.pool = static_cast<uint8_t *>(pool->k);
    a.num_blocks = pool->num_blocks;
    a.n_kv = pool->n_kv;
    a.parents = parents;
    a.beams = beams;
    a.k = k;
    a.tables = block_tables;
    a.W = max_blocks_per_seq;
    a.lens = context_lens;
    a.spare = spare_blocks;
    a.tables_out = tables_out;
    a.lens_out = lens_out;
    a.err = pool->err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)((int64_t)batch * k), (unsigned)pool->n_kv);
    LaunchScope ls(pool, kBlocks, s);
    cudaError_t e = PKV_LAUNCH_BY_POOL(beam_reorder_kernel, grid, s, a);
    ls.done();
    if (e != cudaSuccess) return cuda_fail(e, "paged_beam_reorder launch");
    return PKV_OK;
}
