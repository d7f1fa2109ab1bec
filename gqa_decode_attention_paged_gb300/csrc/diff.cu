// Differential decode attention over the paged cache: one new token per
// sequence.
//
// Mathematics.  KV heads come in pairs p = (2p, 2p + 1).  A pair has two key
// heads K1 = K[2p], K2 = K[2p+1] and one value head of twice the width,
// V = [V[2p] | V[2p+1]].  Each of its G heads has two queries, rows 2h and
// 2h + 1 of the pair's 2 G consecutive query rows:
//   o = softmax(s q1 K1^T) V - lambda softmax(s q2 K2^T) V
//   out = (1 - lambda_init) * w * o / sqrt(mean(o^2) + eps)   (over 2 d channels)
// with lambda = exp(l0 . l1) - exp(l2 . l3) + lambda_init from learned
// vectors.  Both softmax maps are taken over the same positions, so one pass
// over the pair's two cache entries (adjacent in the pool) serves all 2 G
// query rows: they are the columns of the MMAs, column 2h the first map of
// head h and column 2h + 1 its second, and one thread's accumulators hold
// both maps of a head side by side -- the difference and the norm need no
// exchange but a sum over lanes.
//
// What bounds it: HBM, the pair's entries read once (0.75 G MMAs of 16x8x16
// per 512 bytes).  The (sequence, pair, block) stream, its equal slices, the
// per-warp copy rings and the lazy reference maxima are those of decode.cu;
// the difference to it is in the tile: 2 d value channels for every score
// column, and scores of K1 and K2 by separate MMAs over all columns, of which
// each column keeps its own map's (cheaper than zeroing the other's queries:
// the MMA count is the same and nothing is masked).
//
// A run (sequence, pair) that a slice holds whole is finished by its warp.
// Otherwise the warp leaves (m, l, O) for diff_merge_kernel.  A slice cuts at
// most two runs, the one it starts inside of (partial slot 2 * slice) and the
// one it ends inside of (2 * slice + 1), so the workspace grows with the
// number of slices alone, not with batch * heads.
#include <algorithm>
#include <float.h>
#include <math.h>
#include <mutex>

#include "decode_common.cuh"
#include "diff_common.cuh"

namespace pkv {
namespace {

struct DiffArgs {
    int64_t num_blocks;
    int n_kv, n_q, n_pairs;
    const __nv_bfloat16 *q;
    const int32_t *block_tables;
    int W;
    const int32_t *context_lens;
    int batch;
    float qscale;         // scale * log2(e)
    const float *scales;  // FP8: [2 * n_kv]
    DiffWeights w;
    __nv_bfloat16 *out;   // [batch][n_q / 2][2 D]
    float2 *ws_ml;        // [2 * slices][2 G] (reference maximum in log2 units, sum)
    float *ws_o;          // [2 * slices][2 G][2 D], unnormalised
    int slice_blocks;     // blocks per slice; 0 = ceil(total / all warps)
    unsigned *err;
};

// One stage: the pair's two entries, each as decode.cu lays out one.
template <int D, int KV>
struct DGeo {
    static constexpr int E = KV == PKV_BF16 ? 2 : 1;
    static constexpr int ROWB = D * E;
    static constexpr int BOXB = ROWB > 128 ? 128 : ROWB;
    static constexpr int NREG = ROWB / BOXB;
    static constexpr int RGN = kBlockSize * BOXB;
    static constexpr int CSTRIDE = 2 * RGN;         // between column ranges (key then value rows)
    static constexpr int VOFF = RGN;                // value rows after their column range's key rows
    static constexpr int HEAD = 2 * NREG * RGN;     // one KV head's entry
    static constexpr int STAGE = 2 * HEAD;
    static constexpr int BOX_ELEMS = BOXB / E;
};

template <int D, int G, int KV>
struct DCfg {
    using Gm = DGeo<D, KV>;
    // 96 KiB of stages per CTA, two CTAs per SM.  bf16 at d_head 128 (16 KiB a stage): two warps with three
    // stages each; three with two read long contexts of 8 heads a KV head slower (16 x 32768 tokens: 328
    // against 347 us; one sequence of 32768: 41 against 47) and 64 x 1024..2048 tokens no faster (72 us).
    // E4M3 (8 KiB): four with three (256 sequences of 16..4096: 188 us; six with two 195, three with four 191).
    static constexpr int NW = KV == PKV_BF16 && D == 128 ? 2 : 4;
    static constexpr int kThreads = NW * 32;
    static constexpr int kStages = std::min(8, 96 * 1024 / (NW * Gm::STAGE));
    static constexpr int kRing = NW * kStages * Gm::STAGE;
    static constexpr int kBars = kRing;
    static constexpr int kPhys = kBars + NW * kStages * 8;
    static constexpr int kWarpTot = kPhys + NW * kStages * 4;
    static constexpr int kPs = kWarpTot + 4 * NW;
    static size_t smem_bytes(int batch) { return 1024 + (size_t)kPs + 4 * (size_t)(3 * batch + 1); }
};

constexpr float kDiffSlack = 8.0f;  // log2 of the largest weight before the reference maximum is raised

template <int D, int G, int KV>
__global__ void __launch_bounds__(DCfg<D, G, KV>::kThreads, 2)
    diff_decode_kernel(const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ DiffArgs a)
{
    using C = DCfg<D, G, KV>;
    using Gm = typename C::Gm;
    constexpr bool FP8 = KV == PKV_FP8_E4M3;
    constexpr int S = C::kStages, NW = C::NW, NT = D / 16, kThreads = C::kThreads;
    constexpr int COLS = 2 * G;            // query rows of a pair: (head, map)
    constexpr int NB = (COLS + 7) / 8;     // MMA column tiles
    constexpr int CH = NB == 1 ? 2 : 1;    // independent score chains per map and column tile
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g8 = lane >> 2, c4 = lane & 3;
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *ring = smem + warp * S * Gm::STAGE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBars) + warp * S;
    int *phys_st = reinterpret_cast<int *>(smem + C::kPhys) + warp * S;
    int *warp_tot = reinterpret_cast<int *>(smem + C::kWarpTot);
    int32_t *ps = reinterpret_cast<int32_t *>(smem + C::kPs);

    if (tid == 0) {
        prefetch_tensormap(&tm_kv);
        for (int i = 0; i < NW * S; ++i) mbar_init(reinterpret_cast<uint64_t *>(smem + C::kBars) + i, 1);
        fence_mbarrier_init();
    }
    int32_t *cl = ps + a.batch + 1;
    int32_t *rb = cl + a.batch;
    griddep_wait();
    griddep_launch_dependents();
    scan_blocks<NW>(a.context_lens, a.batch, a.W, nullptr, 0, 0, blockIdx.x == 0 ? a.err : nullptr, ps, cl, rb,
                    warp_tot);  // ends with __syncthreads
    Stream st;
    st.ps = ps;
    st.batch = a.batch;
    st.n_kv = a.n_pairs;
    st.total = a.n_pairs * ps[a.batch];
    st.n_warps = (int)gridDim.x * NW;
    st.share = a.slice_blocks > 0 ? a.slice_blocks : max(1, (st.total + st.n_warps - 1) / st.n_warps);
    st.n_slices = (st.total + st.share - 1) / st.share;
    const int me = (int)blockIdx.x * NW + warp;
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {  // empty sequences: zero rows
        if (ps[b + 1] != ps[b]) continue;
        uint4 *o = reinterpret_cast<uint4 *>(a.out + (int64_t)b * a.n_q * D);
        for (int i = tid; i < a.n_q * D / 8; i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
    }

    const uint64_t policy = l2_policy_evict_first();
    bool aborted = false;
    int drain_from = -1;

    // ---- producer (uniform across the warp; lane 0 issues the copies) ----
    auto load_tab = [&](const Seg &s) -> int {
        return s.live && lane < s.n ? a.block_tables[(int64_t)s.p.b * a.W + s.j + lane] : -1;
    };
    Seg cur;
    seg_first(cur, st, me);
    int tab_cur = load_tab(cur);
    Seg nxt = cur;
    seg_next(nxt, st);
    int tab_nxt = load_tab(nxt);
    int seg_k = 0, n_issued = 0;
    auto issue_next = [&]() {
        if (!cur.live) return;
        const int phys = __shfl_sync(kFull, tab_cur, seg_k);
        const int sidx = n_issued % S;
        if (lane == 0) {
            const bool ok = phys >= 0 && phys < a.num_blocks;
            phys_st[sidx] = ok ? phys : -1;
            if (ok) {
                const int y = (int)(((int64_t)phys * a.n_kv + 2 * cur.p.g) * 2 * kBlockSize);
                uint8_t *dst = ring + sidx * Gm::STAGE;
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(&bars[sidx], Gm::STAGE);
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int r = 0; r < Gm::NREG; ++r)
                        tma_load_2d(dst + m * Gm::HEAD + r * Gm::CSTRIDE, &tm_kv, r * Gm::BOX_ELEMS,
                                    y + m * 2 * kBlockSize, &bars[sidx], policy);
            } else {
                atomicOr(a.err, PKV_DEVERR_BLOCK_RANGE);
                mbar_arrive(&bars[sidx]);
            }
        }
        ++n_issued;
        if (++seg_k == cur.n) {
            cur = nxt;
            tab_cur = tab_nxt;
            seg_k = 0;
            seg_next(nxt, st);
            tab_nxt = load_tab(nxt);
        }
    };
    for (int i = 0; i < S; ++i) issue_next();
    const float lam = diff_lambda<D>(a.w, lane);

    const int row_k = (lane & 7) + ((lane >> 3) & 1) * 8, half_k = lane >> 4;
    const int row_v = (lane & 7) + (lane >> 4) * 8, half_v = (lane >> 3) & 1;
    // channel of accumulator rows (tile t, row g8 + 8 i) within a value head
    auto chan = [&](int t, int i) -> int {
        if constexpr (!FP8) return 16 * t + g8 + 8 * i;
        else return 64 * (t >> 2) + 8 * g8 + 4 * ((t >> 1) & 1) + 2 * (t & 1) + i;
    };

    Piece pc;
    bool have = first_piece(st, me, pc);
    int consumed = 0;
    while (have) {
        Piece nx = pc;
        const bool have_nx = next_piece(st, nx);
        // queries as B fragments: thread (g8, c4) holds column 8 nb + g8's pairs of channels
        uint32_t qf[NB][NT][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int col = 8 * nb + g8;
            const bool live = col < COLS;
            const __nv_bfloat16 *qrow = a.q + ((int64_t)pc.b * a.n_q + pc.g * COLS + (live ? col : 0)) * D;
#pragma unroll
            for (int ks = 0; ks < NT; ++ks) {
                if constexpr (!FP8) {
                    qf[nb][ks][0] = live ? *reinterpret_cast<const uint32_t *>(qrow + 16 * ks + 2 * c4) : 0u;
                    qf[nb][ks][1] = live ? *reinterpret_cast<const uint32_t *>(qrow + 16 * ks + 8 + 2 * c4) : 0u;
                } else {  // the order the E4M3 key fragments use, widened to f16 pairs
                    const int d0 = 32 * (ks >> 1) + 8 * c4 + 4 * (ks & 1);
                    const uint2 r = live ? *reinterpret_cast<const uint2 *>(qrow + d0) : make_uint2(0, 0);
                    const float2 x = bf16x2_to_f32x2(r.x), y = bf16x2_to_f32x2(r.y);
                    qf[nb][ks][0] = pack2<true>(x.x, x.y);
                    qf[nb][ks][1] = pack2<true>(y.x, y.y);
                }
            }
        }
        const float qs0 = a.qscale * (FP8 ? a.scales[2 * pc.g] : 1.0f);
        const float qs1 = a.qscale * (FP8 ? a.scales[2 * pc.g + 1] : 1.0f);
        const int C_len = cl[pc.b];
        float o[NB][2 * NT][4];
        float m0[NB], m1[NB], l0[NB], l1[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int t = 0; t < 2 * NT; ++t) o[nb][t][0] = o[nb][t][1] = o[nb][t][2] = o[nb][t][3] = 0.0f;
            m0[nb] = m1[nb] = -FLT_MAX;  // (finite: a score of -inf is below it and weighs 0)
            l0[nb] = l1[nb] = 0.0f;
        }

        for (int j = pc.j0; j < pc.j1; ++j) {
            const int sidx = consumed % S;
            const uint32_t parity = (uint32_t)(consumed / S) & 1u;
            if (!aborted) {
                const bool ok = mbar_wait_bounded(&bars[sidx], parity);
                aborted = __any_sync(kFull, !ok);
                if (aborted) {
                    drain_from = consumed;
                    if (lane == 0) atomicOr(a.err, PKV_DEVERR_TIMEOUT);
                }
            }
            if (!aborted && phys_st[sidx] >= 0) {
                const uint32_t base = smem_u32(ring + sidx * Gm::STAGE);
                const int nv = min(kBlockSize, C_len - j * kBlockSize);
                // ---- scores of both maps, over all columns ----
                float sc[2][CH][NB][4];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
#pragma unroll
                    for (int c = 0; c < CH; ++c)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) sc[m][c][nb][0] = sc[m][c][nb][1] = sc[m][c][nb][2] = sc[m][c][nb][3] = 0.0f;
                    const uint32_t kb = base + m * Gm::HEAD;
                    if constexpr (!FP8) {
#pragma unroll
                        for (int ks = 0; ks < NT; ++ks) {
                            const int chunk = 2 * ks + half_k;
                            uint32_t fa[4];
                            ldsm_x4(kb + (chunk >> 3) * Gm::CSTRIDE + swz<128>(row_k * 128 + (chunk & 7) * 16), fa);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                mma16816<false>(sc[m][ks % CH][nb], fa, qf[nb][ks][0], qf[nb][ks][1]);
                        }
                    } else {
#pragma unroll
                        for (int kk = 0; kk < D / 32; ++kk) {
                            const uint32_t d0 = 32 * kk + 8 * c4;
                            const uint2 x = lds64(kb + swz<Gm::BOXB>(g8 * Gm::ROWB + d0));
                            const uint2 y = lds64(kb + swz<Gm::BOXB>((g8 + 8) * Gm::ROWB + d0));
                            uint32_t f0[4], f1[4];
                            e4m3x4_to_f16x4(x.x, f0[0], f0[2]);
                            e4m3x4_to_f16x4(y.x, f0[1], f0[3]);
                            e4m3x4_to_f16x4(x.y, f1[0], f1[2]);
                            e4m3x4_to_f16x4(y.y, f1[1], f1[3]);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                mma16816<true>(sc[m][0][nb], f0, qf[nb][2 * kk][0], qf[nb][2 * kk][1]);
                                mma16816<true>(sc[m][CH - 1][nb], f1, qf[nb][2 * kk + 1][0], qf[nb][2 * kk + 1][1]);
                            }
                        }
                    }
                }
                // column 2 c4 keeps the first map's scores, column 2 c4 + 1 the second's
                float s[NB][4];
                bool raise = false;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    s[nb][0] = (sc[0][0][nb][0] + (CH == 2 ? sc[0][CH - 1][nb][0] : 0.0f)) * qs0;
                    s[nb][1] = (sc[1][0][nb][1] + (CH == 2 ? sc[1][CH - 1][nb][1] : 0.0f)) * qs1;
                    s[nb][2] = (sc[0][0][nb][2] + (CH == 2 ? sc[0][CH - 1][nb][2] : 0.0f)) * qs0;
                    s[nb][3] = (sc[1][0][nb][3] + (CH == 2 ? sc[1][CH - 1][nb][3] : 0.0f)) * qs1;
                    if (g8 >= nv) s[nb][0] = s[nb][1] = -INFINITY;
                    if (g8 + 8 >= nv) s[nb][2] = s[nb][3] = -INFINITY;
                    raise |= fmaxf(s[nb][0], s[nb][2]) > m0[nb] + kDiffSlack || fmaxf(s[nb][1], s[nb][3]) > m1[nb] + kDiffSlack;
                }
                // ---- raise the reference maxima where a score passes one by the slack ----
                if (__any_sync(kFull, raise)) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        float x0 = fmaxf(s[nb][0], s[nb][2]), x1 = fmaxf(s[nb][1], s[nb][3]);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) {
                            x0 = fmaxf(x0, __shfl_xor_sync(kFull, x0, off));
                            x1 = fmaxf(x1, __shfl_xor_sync(kFull, x1, off));
                        }
                        const float n0 = fmaxf(m0[nb], x0), n1 = fmaxf(m1[nb], x1);
                        const float al0 = ex2_approx(m0[nb] - n0), al1 = ex2_approx(m1[nb] - n1);
                        m0[nb] = n0;
                        m1[nb] = n1;
                        l0[nb] *= al0;
                        l1[nb] *= al1;
#pragma unroll
                        for (int t = 0; t < 2 * NT; ++t) {
                            o[nb][t][0] *= al0;
                            o[nb][t][1] *= al1;
                            o[nb][t][2] *= al0;
                            o[nb][t][3] *= al1;
                        }
                    }
                }
                // P^T: tokens 2c, 2c+1 and 2c+8, 2c+9 of column g8.  bf16 pools: each weight as the sum of
                // two bf16 (16 bits of it), the second taken by a second MMA on the same V fragment.  The
                // difference of the maps is smaller than the maps, so one rounding to bf16 showed in the
                // result (2.6e-3 of it in the 2-norm, against 1.7e-3 now, which the output's own rounding
                // gives); the tensor pipe has room for the extra MMAs (16 sequences of 32768 tokens 2 % slower, 64 of
                // 1024 .. 2048 less than 1 %).
                uint32_t pb[NB][2];
                [[maybe_unused]] uint32_t pl[NB][2];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const float p0 = ex2_approx(s[nb][0] - m0[nb]), p1 = ex2_approx(s[nb][1] - m1[nb]);
                    const float p2 = ex2_approx(s[nb][2] - m0[nb]), p3 = ex2_approx(s[nb][3] - m1[nb]);
                    l0[nb] += p0 + p2;
                    l1[nb] += p1 + p3;
                    const uint32_t w0 = pack2<FP8>(p0, p1), w1 = pack2<FP8>(p2, p3);
                    pb[nb][0] = movm_t(w0);
                    pb[nb][1] = movm_t(w1);
                    if constexpr (!FP8) {
                        const float2 f0 = bf16x2_to_f32x2(w0), f1 = bf16x2_to_f32x2(w1);
                        pl[nb][0] = movm_t(pack2<false>(p0 - f0.x, p1 - f0.y));
                        pl[nb][1] = movm_t(pack2<false>(p2 - f1.x, p3 - f1.y));
                    }
                }
                // masked tokens' values must not reach the MMA (0 * non-finite)
                const uint32_t mk01 = (2 * c4 < nv ? 0x0000ffffu : 0u) | (2 * c4 + 1 < nv ? 0xffff0000u : 0u);
                const uint32_t mk23 = (2 * c4 + 8 < nv ? 0x0000ffffu : 0u) | (2 * c4 + 9 < nv ? 0xffff0000u : 0u);
                // ---- O^T += V^T . P^T, both value heads ----
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t vb = base + m * Gm::HEAD + Gm::VOFF;
                    if constexpr (!FP8) {
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const int chunk = 2 * t + half_v;
                            uint32_t fa[4];
                            ldsm_x4_t(vb + (chunk >> 3) * Gm::CSTRIDE + swz<128>(row_v * 128 + (chunk & 7) * 16), fa);
                            if (nv < kBlockSize) {
                                fa[0] &= mk01;
                                fa[1] &= mk01;
                                fa[2] &= mk23;
                                fa[3] &= mk23;
                            }
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                mma16816<false>(o[nb][m * NT + t], fa, pb[nb][0], pb[nb][1]);
                                mma16816<false>(o[nb][m * NT + t], fa, pl[nb][0], pl[nb][1]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int Q = 0; Q < D / 64; ++Q) {
                            const uint32_t db = 64 * Q + 8 * g8;
                            const uint2 v0 = lds64(vb + swz<Gm::BOXB>((2 * c4) * Gm::ROWB + db));
                            const uint2 v1 = lds64(vb + swz<Gm::BOXB>((2 * c4 + 1) * Gm::ROWB + db));
                            const uint2 v2 = lds64(vb + swz<Gm::BOXB>((2 * c4 + 8) * Gm::ROWB + db));
                            const uint2 v3 = lds64(vb + swz<Gm::BOXB>((2 * c4 + 9) * Gm::ROWB + db));
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t r0 = h ? v0.y : v0.x, r1 = h ? v1.y : v1.x;
                                const uint32_t r2 = h ? v2.y : v2.x, r3 = h ? v3.y : v3.x;
                                uint32_t fa[4], fb[4];
                                e4m3x4_to_f16x4(prmt(r0, r1, 0x5140u), fa[0], fa[1]);
                                e4m3x4_to_f16x4(prmt(r0, r1, 0x7362u), fb[0], fb[1]);
                                e4m3x4_to_f16x4(prmt(r2, r3, 0x5140u), fa[2], fa[3]);
                                e4m3x4_to_f16x4(prmt(r2, r3, 0x7362u), fb[2], fb[3]);
                                if (nv < kBlockSize) {
                                    fa[0] &= mk01; fa[1] &= mk01; fa[2] &= mk23; fa[3] &= mk23;
                                    fb[0] &= mk01; fb[1] &= mk01; fb[2] &= mk23; fb[3] &= mk23;
                                }
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb) {
                                    mma16816<true>(o[nb][m * NT + 4 * Q + 2 * h], fa, pb[nb][0], pb[nb][1]);
                                    mma16816<true>(o[nb][m * NT + 4 * Q + 2 * h + 1], fb, pb[nb][0], pb[nb][1]);
                                }
                            }
                        }
                    }
                }
            }
            __syncwarp();
            ++consumed;
            if (!aborted) issue_next();
        }

        // ---- piece end ----
        const float vs0 = FP8 ? a.scales[a.n_kv + 2 * pc.g] : 1.0f, vs1 = FP8 ? a.scales[a.n_kv + 2 * pc.g + 1] : 1.0f;
        const bool whole = pc.j0 == 0 && pc.j1 == pc.nblk;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float t0 = l0[nb], t1 = l1[nb];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                t0 += __shfl_xor_sync(kFull, t0, off);
                t1 += __shfl_xor_sync(kFull, t1, off);
            }
            const int h = 4 * nb + c4;  // this thread's head of the pair
            if (whole) {
                const float r0 = t0 == 0.0f ? 0.0f : 1.0f / t0, r1 = t1 == 0.0f ? 0.0f : lam / t1;
                float ss = 0.0f;
#pragma unroll
                for (int t = 0; t < 2 * NT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float x = (o[nb][t][2 * i] * r0 - o[nb][t][2 * i + 1] * r1) * (t < NT ? vs0 : vs1);
                        o[nb][t][2 * i] = x;
                        ss = fmaf(x, x, ss);
                    }
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) ss += __shfl_xor_sync(kFull, ss, off);
                const float r = a.w.out_scale * rsqrtf(ss * (1.0f / (2 * D)) + a.w.eps);
                if (h < G) {
                    __nv_bfloat16 *ob = a.out + ((int64_t)pc.b * (a.n_q / 2) + pc.g * G + h) * (2 * D);
#pragma unroll
                    for (int t = 0; t < 2 * NT; ++t)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int d = (t / NT) * D + chan(t % NT, i);
                            const float wt = a.w.norm_weight ? __ldg(a.w.norm_weight + d) : 1.0f;
                            ob[d] = __float2bfloat16_rn(o[nb][t][2 * i] * r * wt);
                        }
                }
            } else if (h < G) {
                const int64_t slot = 2 * (int64_t)pc.slice + (pc.j0 == 0 ? 1 : 0);
                float *wo = a.ws_o + (slot * COLS + 2 * h) * (2 * D);
#pragma unroll
                for (int t = 0; t < 2 * NT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int d = (t / NT) * D + chan(t % NT, i);
                        const float vs = t < NT ? vs0 : vs1;
                        wo[d] = o[nb][t][2 * i] * vs;
                        wo[2 * D + d] = o[nb][t][2 * i + 1] * vs;
                    }
                if (g8 == 0) {
                    float2 *ml = a.ws_ml + slot * COLS + 2 * h;
                    ml[0] = make_float2(m0[nb], t0);
                    ml[1] = make_float2(m1[nb], t1);
                }
            }
        }
        pc = nx;
        have = have_nx;
    }

    if (drain_from >= 0)  // copies may still be in flight only after a timeout
        for (int k = drain_from; k < n_issued; ++k)
            mbar_wait_bounded(&bars[k % S], (uint32_t)(k / S) & 1u, 100000000ull);
}

// ---------------------------------------------------------------------------
// Merge of the runs that slices cut: each head's two maps by log-sum-exp over
// the pieces in slice order, then the difference and the norm.
// ---------------------------------------------------------------------------

constexpr int kDiffMergeWarps = 8;

template <int D, int G>
__global__ void __launch_bounds__(kDiffMergeWarps * 32, 2) diff_merge_kernel(const __grid_constant__ DiffArgs a, int n_warps)
{
    constexpr int COLS = 2 * G;
    constexpr int KW = D / 32;   // 16-byte chunks a lane holds of a head's two rows of 2 D numbers
    constexpr int HK = KW / 2;   // the first HK are the first map's
    constexpr int PB = 16 / KW;  // pieces in flight
    constexpr int NWM = kDiffMergeWarps;
    extern __shared__ int32_t ps[];  // [batch + 1]
    __shared__ int warp_tot[NWM];
    __shared__ float4 part[NWM][KW][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    scan_blocks<NWM>(a.context_lens, a.batch, a.W, nullptr, 0, 0, nullptr, ps, nullptr, nullptr, warp_tot);
    const int total = a.n_pairs * ps[a.batch];
    const int share = a.slice_blocks > 0 ? a.slice_blocks : max(1, (total + n_warps - 1) / n_warps);
    const float lam = diff_lambda<D>(a.w, lane);
    griddep_wait();  // the decode kernel's partials
    griddep_launch_dependents();
    const int64_t items = (int64_t)a.batch * a.n_pairs * G;  // (sequence, pair, head)
    const bool shared = items <= gridDim.x;  // a CTA per item, its pieces dealt to the warps; else a warp per item
    const int64_t first = shared ? blockIdx.x : (int64_t)blockIdx.x * NWM + warp;
    const int64_t step = shared ? gridDim.x : (int64_t)gridDim.x * NWM;
    const int w0 = shared ? warp : 0, nw = shared ? NWM : 1;
    for (int64_t it = first; it < items; it += step) {
        const int h = (int)(it % G);
        const int p = (int)(it / G % a.n_pairs), b = (int)(it / ((int64_t)G * a.n_pairs));
        const int nblk = ps[b + 1] - ps[b];
        if (nblk == 0) continue;
        const int start = a.n_pairs * ps[b] + p * nblk;
        const int s0 = start / share;
        const int np = (start + nblk - 1) / share - s0 + 1;
        if (np <= 1) continue;  // finished by the decode kernel
        // piece k lies in slice s0 + k; the first began at the run's start
        auto slot = [&](int k) -> int64_t { return 2 * (int64_t)(s0 + k) + (k == 0 ? 1 : 0); };
        auto ml_of = [&](int k) -> float4 {  // (m, l) of the two maps
            return __ldcg(reinterpret_cast<const float4 *>(a.ws_ml + slot(k) * COLS + 2 * h));
        };
        float4 buf[PB][KW];
        float4 bml[PB];
        auto fetch = [&](int i, int k) {
            const float4 *src = reinterpret_cast<const float4 *>(a.ws_o + (slot(k) * COLS + 2 * h) * (2 * D));
#pragma unroll
            for (int c = 0; c < KW; ++c) buf[i][c] = __ldcg(src + lane + 32 * c);
            bml[i] = ml_of(k);
        };
#pragma unroll
        for (int i = 0; i < PB; ++i)
            if (w0 + i * nw < np) fetch(i, w0 + i * nw);
        float M0 = -INFINITY, L0 = 0.0f, M1 = -INFINITY, L1 = 0.0f;
        for (int k = lane; k < np; k += 32) {
            const float4 v = ml_of(k);
            const float n0 = fmaxf(M0, v.x), n1 = fmaxf(M1, v.z);
            L0 = n0 == -INFINITY ? L0 + v.y : L0 * exp2f(M0 - n0) + v.y * exp2f(v.x - n0);
            L1 = n1 == -INFINITY ? L1 + v.w : L1 * exp2f(M1 - n1) + v.w * exp2f(v.z - n1);
            M0 = n0;
            M1 = n1;
        }
        float T0 = M0, T1 = M1;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            T0 = fmaxf(T0, __shfl_xor_sync(kFull, T0, o));
            T1 = fmaxf(T1, __shfl_xor_sync(kFull, T1, o));
        }
        // a map none of whose positions could be read (bad block ids) weighs nothing
        L0 = M0 == -INFINITY ? L0 : L0 * exp2f(M0 - T0);
        L1 = M1 == -INFINITY ? L1 : L1 * exp2f(M1 - T1);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            L0 += __shfl_xor_sync(kFull, L0, o);
            L1 += __shfl_xor_sync(kFull, L1, o);
        }
        float4 acc[KW];
#pragma unroll
        for (int c = 0; c < KW; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = w0; k0 < np; k0 += PB * nw) {
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                const int k = k0 + i * nw;
                if (k < np) {
                    const float e0 = bml[i].x == -INFINITY ? 0.0f : exp2f(bml[i].x - T0);
                    const float e1 = bml[i].z == -INFINITY ? 0.0f : exp2f(bml[i].z - T1);
#pragma unroll
                    for (int c = 0; c < KW; ++c) {
                        const float e = c < HK ? e0 : e1;
                        acc[c].x = fmaf(e, buf[i][c].x, acc[c].x);
                        acc[c].y = fmaf(e, buf[i][c].y, acc[c].y);
                        acc[c].z = fmaf(e, buf[i][c].z, acc[c].z);
                        acc[c].w = fmaf(e, buf[i][c].w, acc[c].w);
                    }
                    if (k + PB * nw < np) fetch(i, k + PB * nw);
                }
            }
        }
        if (shared) {  // the warps' sums, added in warp order (one item per CTA: uniform branch)
#pragma unroll
            for (int c = 0; c < KW; ++c) part[warp][c][lane] = acc[c];
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int c = 0; c < KW; ++c)
                    for (int w = 1; w < NWM; ++w) {
                        const float4 y = part[w][c][lane];
                        acc[c].x += y.x;
                        acc[c].y += y.y;
                        acc[c].z += y.z;
                        acc[c].w += y.w;
                    }
            }
        }
        if (!shared || warp == 0) {
            const float r0 = L0 == 0.0f ? 0.0f : 1.0f / L0, r1 = L1 == 0.0f ? 0.0f : lam / L1;
            float ss = 0.0f;
#pragma unroll
            for (int c = 0; c < HK; ++c) {
                float4 &x = acc[c];
                const float4 y = acc[c + HK];
                x.x = x.x * r0 - y.x * r1;
                x.y = x.y * r0 - y.y * r1;
                x.z = x.z * r0 - y.z * r1;
                x.w = x.w * r0 - y.w * r1;
                ss += x.x * x.x + x.y * x.y + x.z * x.z + x.w * x.w;
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
            const float r = a.w.out_scale * rsqrtf(ss * (1.0f / (2 * D)) + a.w.eps);
            __nv_bfloat16 *ob = a.out + ((int64_t)b * (a.n_q / 2) + p * G + h) * (2 * D);
#pragma unroll
            for (int c = 0; c < HK; ++c) {
                const int d = 4 * (lane + 32 * c);
                const float4 wt = a.w.norm_weight ? __ldg(reinterpret_cast<const float4 *>(a.w.norm_weight + d))
                                                  : make_float4(1.f, 1.f, 1.f, 1.f);
                *reinterpret_cast<uint2 *>(ob + d) = make_uint2(pack2<false>(acc[c].x * r * wt.x, acc[c].y * r * wt.y),
                                                                pack2<false>(acc[c].z * r * wt.z, acc[c].w * r * wt.w));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

constexpr int kMergeResident = 2;  // merge CTAs per SM (4: 72.1 us at 64 x 1024..2048 tokens, 2: 71.8)
// Blocks a warp should have before another is used.  One: a short sequence is bound by the chain of its warps
// (300 tokens: 10.3 us; with 2 blocks 11.1, with 4 12.2).
constexpr int kDiffMinBlocks = 1;

constexpr int kMaxDevices = 64;

// Resident CTAs per SM of the decode kernel at this batch (found once per
// device and 1024 sequences, whose lists share the SM's shared memory).
template <int D, int G, int KV>
pkv_status resident(const pkv_pool *pool, int batch, int *occ)
{
    using C = DCfg<D, G, KV>;
    auto kern = diff_decode_kernel<D, G, KV>;
    static std::mutex mu;
    static int8_t known[kMaxDevices][kMaxBatch / 1024 + 1];  // 0: not yet
    const int step = (batch + 1023) / 1024;
    std::lock_guard<std::mutex> lock(mu);
    int8_t *k = pool->device < kMaxDevices ? &known[pool->device][step] : nullptr;
    if (!k || *k == 0) {
        int optin = 0, n = 0;
        cudaError_t e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, pool->device);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, optin);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(diff_merge_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     4 * (kMaxBatch + 1));
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, C::kThreads, C::smem_bytes(step * 1024));
        if (e != cudaSuccess) return cuda_fail(e, "paged_diff_decode_attention: kernel attributes");
        if (n < 1) return fail(PKV_EUNSUPPORTED, "paged_diff_decode_attention: the kernel does not fit on an SM");
        *occ = n;
        if (k) *k = (int8_t)n;
        return PKV_OK;
    }
    *occ = *k;
    return PKV_OK;
}

// The decode grid, and the workspace of a call on it: partials of two runs per
// slice, (m, l) first.
struct Plan {
    int grid = 0;
    size_t ml_bytes = 0, bytes = 0;
};

// `most_resident`: for any number of sequences up to `batch`.  Every part of the plan rises with the batch but the
// resident CTAs, whose shared memory holds the batch's lists: the fewest sequences have the most of them.
template <int D, int G, int KV>
pkv_status plan_call(const pkv_pool *pool, int batch, int W, Plan *pl, bool most_resident = false)
{
    using C = DCfg<D, G, KV>;
    int occ = 0;
    pkv_status st = resident<D, G, KV>(pool, most_resident ? 1 : batch, &occ);
    if (st != PKV_OK) return st;
    const int slice_blocks = pool->partition_tokens / kBlockSize;
    const int64_t most = (int64_t)batch * (pool->n_kv / 2) * W;  // blocks of the largest possible batch
    const int64_t want = (most + (int64_t)C::NW * kDiffMinBlocks - 1) / ((int64_t)C::NW * kDiffMinBlocks);
    pl->grid = (int)std::max<int64_t>(1, std::min<int64_t>((int64_t)pool->num_sms * occ, want));
    const int64_t slices = slice_blocks > 0 ? (most + slice_blocks - 1) / slice_blocks : (int64_t)pl->grid * C::NW;
    pl->ml_bytes = ((size_t)slices * 2 * 2 * G * sizeof(float2) + 255) & ~size_t(255);
    pl->bytes = pl->ml_bytes + (size_t)slices * 2 * 2 * G * 2 * D * sizeof(float);
    return PKV_OK;
}

template <int D, int G, int KV>
pkv_status launch(pkv_pool *pool, DiffArgs a, cudaStream_t s)
{
    using C = DCfg<D, G, KV>;
    Plan pl;
    pkv_status st = plan_call<D, G, KV>(pool, a.batch, a.W, &pl);
    if (st != PKV_OK) return st;
    st = ensure_workspace(pool, pl.bytes, s, "paged_diff_decode_attention");
    if (st != PKV_OK) return st;
    a.ws_ml = static_cast<float2 *>(pool->ws);
    a.ws_o = reinterpret_cast<float *>(static_cast<uint8_t *>(pool->ws) + pl.ml_bytes);
    cudaError_t e;
    {
        LaunchScope ls(pool, kDecode, s);
        e = launch_pdl(diff_decode_kernel<D, G, KV>, dim3(pl.grid), dim3(C::kThreads), C::smem_bytes(a.batch), s,
                       pool->tm_entry, a);
        ls.done();
        if (e != cudaSuccess) return cuda_fail(e, "paged_diff_decode_attention launch");
    }
    // merge: a CTA per (sequence, pair, head) while that many are resident, else a warp each
    const int64_t items = (int64_t)a.batch * a.n_pairs * G;
    const int mgrid = (int)std::min<int64_t>(items, (int64_t)pool->num_sms * kMergeResident);
    LaunchScope ls(pool, kMerge, s);
    e = launch_pdl(diff_merge_kernel<D, G>, dim3(mgrid), dim3(kDiffMergeWarps * 32), 4 * ((size_t)a.batch + 1), s, a,
                   pl.grid * C::NW);
    ls.done();
    if (e != cudaSuccess) return cuda_fail(e, "paged_diff_decode_attention: merge launch");
    return PKV_OK;
}

// Run f<D, G, KV> for the pool's head size and type and this group size.
template <template <int, int, int> class F, typename... A>
pkv_status for_config(const pkv_pool *pool, int G, A &&...args)
{
#define PKV_G(D, KV)                                          \
    switch (G) {                                              \
    case 1: return F<D, 1, KV>::run(std::forward<A>(args)...); \
    case 2: return F<D, 2, KV>::run(std::forward<A>(args)...); \
    case 4: return F<D, 4, KV>::run(std::forward<A>(args)...); \
    case 8: return F<D, 8, KV>::run(std::forward<A>(args)...); \
    }
    if (pool->d_head == 128) {
        if (pool->dtype == PKV_BF16) { PKV_G(128, PKV_BF16) } else { PKV_G(128, PKV_FP8_E4M3) }
    } else {
        if (pool->dtype == PKV_BF16) { PKV_G(64, PKV_BF16) } else { PKV_G(64, PKV_FP8_E4M3) }
    }
#undef PKV_G
    return fail(PKV_EUNSUPPORTED, "differential decode: group size %d unsupported (1, 2, 4 or 8)", G);
}

template <int D, int G, int KV>
struct Launch {
    static pkv_status run(pkv_pool *pool, const DiffArgs &a, cudaStream_t s) { return launch<D, G, KV>(pool, a, s); }
};

template <int D, int G, int KV>
struct PlanMost {
    static pkv_status run(const pkv_pool *pool, int batch, int W, Plan *pl)
    {
        return plan_call<D, G, KV>(pool, batch, W, pl, true);
    }
};

}  // namespace

pkv_status check_diff_pool(const pkv_pool *pool, const char *who)
{
    if (pool->dtype == PKV_INT4) return fail(PKV_EUNSUPPORTED, "%s: bf16 and FP8 pools only (not 4-bit)", who);
    if (pool->n_kv % 2) return fail(PKV_EUNSUPPORTED, "%s: the pool's KV heads (%d) do not come in pairs", who, pool->n_kv);
    return PKV_OK;
}

pkv_status check_diff_args(const pkv_pool *pool, const char *who, const pkv_diff_params *params, DiffWeights *w)
{
    pkv_status st = check_diff_pool(pool, who);
    if (st != PKV_OK) return st;
    if (!params) return fail(PKV_EINVAL, "%s: NULL params", who);
    if (!params->lambdas) return fail(PKV_EINVAL, "%s: NULL lambdas", who);
    if (((uintptr_t)params->lambdas & 3u) || ((uintptr_t)params->norm_weight & 15u))
        return fail(PKV_EINVAL, "%s: lambdas must be 4-byte and norm_weight 16-byte aligned", who);
    if (!isfinite(params->lambda_init)) return fail(PKV_EINVAL, "%s: lambda_init is not finite", who);
    if (!(params->eps > 0.0f) || !isfinite(params->eps)) return fail(PKV_EINVAL, "%s: eps must be finite and above 0", who);
    w->lambdas = params->lambdas;
    w->norm_weight = params->norm_weight;
    w->lambda_init = params->lambda_init;
    w->out_scale = 1.0f - params->lambda_init;
    w->eps = params->eps;
    return PKV_OK;
}

}  // namespace pkv

using namespace pkv;

extern "C" pkv_status paged_diff_decode_attention(pkv_pool *pool, const void *q, int32_t n_q,
                                                  const int32_t *block_tables, int32_t max_blocks_per_seq,
                                                  const int32_t *context_lens, int32_t batch, float scale,
                                                  const pkv_diff_params *params, void *out, void *stream)
{
    const char *who = "paged_diff_decode_attention";
    pkv_status st = check_step_args(pool, who, n_q, max_blocks_per_seq, batch, scale);
    DiffArgs a;
    if (st == PKV_OK) st = check_diff_args(pool, who, params, &a.w);
    if (st != PKV_OK || batch == 0) return st;
    if (!q || !block_tables || !context_lens || !out) return fail(PKV_EINVAL, "%s: NULL device pointer", who);
    if (((uintptr_t)q | (uintptr_t)out) & 15u) return fail(PKV_EINVAL, "%s: q and out must be 16-byte aligned", who);
    if (((uintptr_t)block_tables | (uintptr_t)context_lens) & 3u)
        return fail(PKV_EINVAL, "%s: tables and lengths must be 4-byte aligned", who);
    st = check_pool_device(pool, who);
    if (st != PKV_OK) return st;
    a.num_blocks = pool->num_blocks;
    a.n_kv = pool->n_kv;
    a.n_q = n_q;
    a.n_pairs = pool->n_kv / 2;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.block_tables = block_tables;
    a.W = max_blocks_per_seq;
    a.context_lens = context_lens;
    a.batch = batch;
    a.qscale = scale * kLog2e;
    a.scales = pool->scales;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.ws_ml = nullptr;
    a.ws_o = nullptr;
    a.slice_blocks = pool->partition_tokens / kBlockSize;
    a.err = pool->err;
    return for_config<Launch>(pool, n_q / pool->n_kv, pool, a, static_cast<cudaStream_t>(stream));
}

extern "C" pkv_status paged_diff_reserve_workspace(pkv_pool *pool, int32_t batch, int32_t n_q,
                                                   int32_t max_blocks_per_seq)
{
    const char *who = "paged_diff_reserve_workspace";
    pkv_status st = check_step_args(pool, who, n_q, max_blocks_per_seq, batch, 1.0f);
    if (st == PKV_OK) st = check_diff_pool(pool, who);
    if (st != PKV_OK || batch == 0) return st;
    st = check_pool_device(pool, who);
    size_t bytes = 0;
    for (int G = 1; st == PKV_OK && G <= n_q / pool->n_kv; G *= 2) {  // fewer query heads, too
        Plan pl;
        st = for_config<PlanMost>(pool, G, pool, batch, max_blocks_per_seq, &pl);
        bytes = std::max(bytes, pl.bytes);
    }
    return st == PKV_OK ? ensure_workspace(pool, bytes) : st;
}
