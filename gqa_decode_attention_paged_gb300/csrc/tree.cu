// Attention of a tree of drafted tokens over the paged cache.
//
// Mathematics.  Node i of sequence b (row r = qo_indptr[b] + i) sits at cached
// position C - T + i; for query head h of KV head g
//   out = sum_p softmax_p(s q_rh . K_pg) V_pg
// over the positions before the nodes and the nodes j whose bit is set in row
// r's mask.  One pass over the keys with a running maximum and sum.
//
// A first form: one thread block per (row, KV head), its warps on every fourth
// key, a lane on D / 32 channels.
#include <float.h>

#include "pkv_internal.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;

struct Args {
    const uint8_t *pool;
    int64_t num_blocks, n_rows;
    int n_q, n_kv;
    const __nv_bfloat16 *q;
    const int32_t *qo_indptr;
    const uint64_t *mask;
    int words;
    const int32_t *block_tables;
    int W;
    const int32_t *context_lens;
    int batch;
    float qscale;         // scale * log2(e)
    const float *scales;  // FP8 pools: [2 * n_kv]
    __nv_bfloat16 *out;
    unsigned *err;
};

template <int D, int G, bool F8>
__global__ void __launch_bounds__(kWarps * 32) tree_kernel(const __grid_constant__ Args a)
{
    constexpr int PL = D / 32;  // channels of a lane
    constexpr int KV = F8 ? PKV_FP8_E4M3 : PKV_BF16;
    constexpr int ROWB = (int)kv_row_bytes(KV, D);
    __shared__ float sm[kWarps][G], sl[kWarps][G], so[kWarps][G][D];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;
    const int g = blockIdx.y;
    if (row == 0 && g == 0)
        for (int b = threadIdx.x; b < a.batch; b += kWarps * 32)
            if (a.qo_indptr[b] < 0 || a.qo_indptr[b + 1] < a.qo_indptr[b]) atomicOr(a.err, PKV_DEVERR_CTX_RANGE);
    int lo = 0, hi = a.batch;  // the last sequence that begins at or before the row
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.qo_indptr[mid] <= row) lo = mid; else hi = mid;
    }
    const int64_t first = a.qo_indptr[lo], end = a.qo_indptr[lo + 1];
    if (first < 0 || row < first || row >= end) return;
    const int64_t T = end - first;
    const int C = a.context_lens[lo];
    if (end > a.n_rows || T > 64 * a.words || C < T || C > a.W * kBlockSize) {
        if (threadIdx.x == 0) atomicOr(a.err, PKV_DEVERR_CTX_RANGE);
        return;
    }
    const int base = C - (int)T;
    float q[G][PL], m[G], l[G], o[G][PL];
    const float qs = a.qscale * (F8 ? a.scales[g] : 1.0f), vs = F8 ? a.scales[a.n_kv + g] : 1.0f;
#pragma unroll
    for (int h = 0; h < G; ++h) {
        m[h] = -FLT_MAX;  // (finite: a score of -inf is below it and weighs 0)
        l[h] = 0.0f;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            q[h][i] = __bfloat162float(a.q[(row * a.n_q + g * G + h) * D + lane * PL + i]);
            o[h][i] = 0.0f;
        }
    }
    auto elem = [&](const uint8_t *p, int i) -> float {
        if constexpr (F8) return (float)reinterpret_cast<const __nv_fp8_e4m3 *>(p)[i];
        else return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
    };
    for (int pos = warp; pos < C; pos += kWarps) {
        if (pos >= base) {
            const int j = pos - base;
            if (!((a.mask[row * a.words + j / 64] >> (j % 64)) & 1)) continue;
        }
        const int32_t blk = a.block_tables[(int64_t)lo * a.W + pos / kBlockSize];
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) atomicOr(a.err, PKV_DEVERR_BLOCK_RANGE);
            continue;
        }
        const uint8_t *k = a.pool + ((int64_t)blk * a.n_kv + g) * kv_entry_bytes(KV, D) + pos % kBlockSize * ROWB;
        const uint8_t *v = k + kBlockSize * ROWB;
        float kf[PL], vf[PL];
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            kf[i] = elem(k, lane * PL + i);
            vf[i] = elem(v, lane * PL + i);
        }
#pragma unroll
        for (int h = 0; h < G; ++h) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < PL; ++i) s = fmaf(q[h][i], kf[i], s);
#pragma unroll
            for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(kFull, s, x);
            s *= qs;
            const float mn = fmaxf(m[h], s), f = exp2f(m[h] - mn), w = exp2f(s - mn);
            l[h] = l[h] * f + w;
#pragma unroll
            for (int i = 0; i < PL; ++i) o[h][i] = o[h][i] * f + w * vf[i];
            m[h] = mn;
        }
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
        sm[warp][h] = m[h];
        sl[warp][h] = l[h];
#pragma unroll
        for (int i = 0; i < PL; ++i) so[warp][h][lane * PL + i] = o[h][i];
    }
    __syncthreads();
    for (int h = warp; h < G; h += kWarps) {
        float M = -FLT_MAX, L = 0.0f, acc[PL] = {};
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w][h]);
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(sm[w][h] - M);
            L += sl[w][h] * f;
#pragma unroll
            for (int i = 0; i < PL; ++i) acc[i] += so[w][h][lane * PL + i] * f;
        }
        const float inv = L == 0.0f ? 0.0f : vs / L;
#pragma unroll
        for (int i = 0; i < PL; ++i)
            a.out[(row * a.n_q + g * G + h) * D + lane * PL + i] = __float2bfloat16(acc[i] * inv);
    }
}

template <int D, bool F8>
cudaError_t launch(const Args &a, int G, cudaStream_t s)
{
    const dim3 grid((unsigned)a.n_rows, (unsigned)a.n_kv);
    switch (G) {
    case 1: return launch_pdl(tree_kernel<D, 1, F8>, grid, dim3(kWarps * 32), 0, s, a);
    case 2: return launch_pdl(tree_kernel<D, 2, F8>, grid, dim3(kWarps * 32), 0, s, a);
    case 4: return launch_pdl(tree_kernel<D, 4, F8>, grid, dim3(kWarps * 32), 0, s, a);
    default: return launch_pdl(tree_kernel<D, 8, F8>, grid, dim3(kWarps * 32), 0, s, a);
    }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status paged_tree_attention(pkv_pool *pool, const void *q, int64_t n_rows, int32_t n_q,
                                           const int32_t *qo_indptr, const uint64_t *tree_mask, int32_t mask_words,
                                           const int32_t *block_tables, int32_t max_blocks_per_seq,
                                           const int32_t *context_lens, int32_t batch, float scale, void *out,
                                           void *stream)
{
    const char *who = "paged_tree_attention";
    pkv_status st = check_step_args(pool, who, n_q, max_blocks_per_seq, batch, scale);
    if (st != PKV_OK) return st;
    if (pool->dtype == PKV_INT4) return fail(PKV_EUNSUPPORTED, "%s: bf16 and FP8 pools only (not 4-bit)", who);
    if (n_rows < 0) return fail(PKV_EINVAL, "%s: n_rows < 0", who);
    if (mask_words < 1) return fail(PKV_EINVAL, "%s: mask_words %d", who, mask_words);
    if (mask_words > 16) return fail(PKV_EUNSUPPORTED, "%s: mask_words %d > 16", who, mask_words);
    if (batch == 0 || n_rows == 0) return PKV_OK;
    const int G = n_q / pool->n_kv;
    if (n_rows > INT32_MAX / G) return fail(PKV_EUNSUPPORTED, "%s: more than 2^31 query rows x group size", who);
    if (!q || !qo_indptr || !tree_mask || !block_tables || !context_lens || !out)
        return fail(PKV_EINVAL, "%s: NULL device pointer", who);
    if (((uintptr_t)q & 15u) || ((uintptr_t)out & 31u))
        return fail(PKV_EINVAL, "%s: q must be 16-byte and out 32-byte aligned", who);
    if (((uintptr_t)qo_indptr | (uintptr_t)block_tables | (uintptr_t)context_lens) & 3u || ((uintptr_t)tree_mask & 7u))
        return fail(PKV_EINVAL, "%s: indptr, tables and lengths must be 4-byte, masks 8-byte aligned", who);
    st = check_pool_device(pool, who);
    if (st != PKV_OK) return st;
    Args a;
    a.pool = static_cast<const uint8_t *>(pool->k);
    a.num_blocks = pool->num_blocks;
    a.n_rows = n_rows;
    a.n_q = n_q;
    a.n_kv = pool->n_kv;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.qo_indptr = qo_indptr;
    a.mask = tree_mask;
    a.words = mask_words;
    a.block_tables = block_tables;
    a.W = max_blocks_per_seq;
    a.context_lens = context_lens;
    a.batch = batch;
    a.qscale = scale * kLog2e;
    a.scales = pool->scales;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.err = pool->err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f8 = pool->dtype == PKV_FP8_E4M3;
    LaunchScope ls(pool, kDecode, s);
    cudaError_t e = pool->d_head == 128 ? (f8 ? launch<128, true>(a, G, s) : launch<128, false>(a, G, s))
                                        : (f8 ? launch<64, true>(a, G, s) : launch<64, false>(a, G, s));
    ls.done();
    if (e != cudaSuccess) return cuda_fail(e, "paged_tree_attention launch");
    return PKV_OK;
}
