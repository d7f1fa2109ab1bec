// Differential attention of a chunk of new tokens over the paged cache, on the
// tcgen05 tensor cores.
//
// Mathematics (see diff.cu for the head layout): for the rows of a pair's G
// heads, o = (P1 - lambda P2) V with P_m = softmax(s Q_m K_m^T) and V the
// pair's two value heads side by side.  A first sweep over the keys finds each
// row's maximum m and sum l of both maps; a second one recomputes the scores,
// forms ONE weight per key,
//   w = c1 2^(s1 - m1) -+ c2 2^(s2 - m2),   c1 / c2 = l2 / (|lambda| l1),
// the larger of c1, c2 being 2^8 (weights stay within f16's range whatever
// the two sums are), and adds w V; o = accumulator / (c1 l1).  The difference
// is taken in fp32 before the rounding to the product's type, so what the two
// maps share never enters it, and V is multiplied once instead of once per
// map.  That rounding is to bf16 (bf16 pools: V's range is not f16's), which
// makes the result's 2-norm error 2.3e-3 where its own rounding alone is 1.7e-3
// (a second bf16 for what is left, as in diff.cu, would be a third more MMA
// work), or to f16 (FP8 pools: 1.7e-3).  With the second Q K^T the MMA work is
// that of separate products of both maps (12 d per row and key), in half the
// accumulator -- two accumulators of 2 d columns would take all of tensor memory
// at d_head 128 and leave none for scores (at d_head 64 they would not; one
// sweep there is not built).  All statistics are final before the first weight
// is formed: no accumulator is ever rescaled.
//
// Design (persistent clusters of two CTAs, one per SM, warp-specialised; the
// times are of 16 prompts of 700..1024 tokens on contexts of up to 2048, bf16,
// d_head 128, 32 query heads: 369 us in all, 200 for the MMAs alone; pairs of
// times compare two forms at the state when the choice was made):
//   * a tile is 128 query rows (token, head) of one (sequence, pair): both
//     maps' queries.  A step is 128 keys.  The two CTAs of a cluster take
//     neighbouring tiles of the same (sequence, pair) and walk the same keys at
//     about the same time, each copying for itself (the second read of a unit
//     comes from the L2).  A step moves 6 units of 32 KiB into each SM.  Both
//     walk to the second tile's last key: where each stops at its own, they fall
//     out of step and their reads no longer meet (478 us against 369).
//   * warp 16 streams Q and, through one ring, what the MMAs take in the order
//     they take it: K_m units (128 keys of one map) and, in the second sweep, V
//     units (64 keys x 2 d channels).  One ring for both: in the first sweep
//     all of it holds keys.
//   * warp 17 issues the MMAs of the scores, another warp those of the products,
//     each as one warp from uniform registers (from inside a lane's branch an
//     MMA took 80 cycles to issue, 640 a unit, and that bound the kernel).
//     The first sweep alternates between the maps' scores.  In the second one
//     the halves of a step (64 keys) are half a step apart, so that one half's
//     weights are formed while the tensor cores work for the other, although
//     scores and weights have one place each: S_2 of the next step follows as
//     soon as this one's is in registers, S_1 of its halves when the products
//     of this one's are done.  One warp for all of it held products back behind
//     the scores' waits (397 us against 377).
//   * the warps after that prepare units: value rows behind the sequence's end
//     are zeroed, and FP8 units are widened to f16 in place, by four warps (two
//     bound the kernel: 596 us against 504 at d_head 128).  Widening writes and
//     reads shared memory once more than the MMAs alone, which keep it busy as
//     it is: FP8 prompts at d_head 128 take 455 us.
//   * sixteen warps work on scores, four threads a row (a step's exponentials
//     are many, and short dependent chains need several warps per scheduler to
//     fill it: with eight warps a step took twice as long).  First sweep: each
//     keeps (m, l) of one map and one half of every step's keys; second sweep:
//     each forms the weights of 32 keys of a step from both maps' scores, over
//     which the weights are written; at the end each holds a quarter of its
//     row of O.  The four threads swap statistics, and later sums of squares,
//     through columns of O that are not in use at that moment.
//   * value rows behind the sequence's end (a page that ends inside a tile)
//     are zeroed in shared memory before their product: a weight of 0 does not
//     cancel what is not finite.
//   * few rows (kRange): when the call's tiles would leave most SMs idle (a few
//     drafted tokens on long caches), a cluster of 2 to 16 CTAs takes one tile,
//     a range of its keys each.  Between the sweeps every CTA reads the others'
//     statistics (distributed shared memory), so all form their weights with
//     the row's final factors, and at the end the parts of o are plain sums:
//     each CTA adds, in order, and normalises its share of the rows.
// Every mbarrier wait is bounded; on a timeout the CTA records
// PKV_DEVERR_TIMEOUT, every role stops, the MMA and copy pipes are drained
// (bounded) and the tensor memory is released before the CTA exits.
#include <algorithm>
#include <climits>
#include <mutex>
#include <type_traits>

#include "diff_common.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kRows = 128;  // query rows per tile (= TMEM lanes)
constexpr int kKeys = 128;  // keys per step
constexpr int kStepBlocks = kKeys / kBlockSize;
constexpr int kVKeys = 64;  // keys of a V unit
constexpr int kUnitBlocks = kVKeys / kBlockSize;
constexpr int kSoftmaxWarps = 16;
constexpr int kCopyWarp = 16, kScoreWarp = 17, kPrepWarp = 18;
template <bool F8>
struct Warps {
    static constexpr int kPreps = F8 ? 4 : 1;  // warps kPrepWarp .. make units ready
    static constexpr int kProduct = kPrepWarp + kPreps;
    static constexpr int kThreads = (F8 ? 24 : 20) * 32;
    // FP8 pools: registers a thread at the launch, then of the warps on scores and of the others
    static constexpr int kLaunchRegs = 80, kScoreRegs = 96, kWorkRegs = 48;
    static_assert(kSoftmaxWarps * kScoreRegs + (24 - kSoftmaxWarps) * kWorkRegs <= 24 * kLaunchRegs,
                  "more registers than the launch has");
};
// Tensor memory: S_1 at 0, S_2 at 128 (fp32 scores of 128 keys; the weights of keys 32 g .. + 31, packed in
// pairs, over the first 16 columns of their S_1), O at 256 (2 d).  While a tile has no product in O yet, its
// columns kColStat + 2 g hold thread g's (m, l); when O is in registers, the first column of each thread's
// quarter holds its sum of squares (neither place is the other's).
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256, kColStat = kColO + 8;
constexpr uint32_t kKHalf = kKeys * 128;   // a 64-column range of a Q or K tile
constexpr uint32_t kVChunk = kVKeys * 128; // a 64-channel range of a V unit
constexpr float kBoost = 8.0f;             // log2 of the larger of c1, c2

struct Args {
    const int32_t *qo_indptr;  // [batch + 1]
    const int32_t *block_tables;
    int W;
    const int32_t *context_lens;
    int batch, n_q, n_kv, n_pairs;
    int window;           // sequences whose tiles are ordered among themselves (32 at most)
    int64_t num_blocks, n_rows;
    int oob_row;          // a row index past the end of the pool's entry rows (zero-filled box)
    float qscale;         // scale * log2(e)
    const float *scales;  // FP8 pools: [2 * n_kv] fp32, K scales then V scales
    DiffWeights w;
    __nv_bfloat16 *out;   // [n_rows][n_q / 2][2 D]
    unsigned *err;
};

// What a cluster does: two CTAs a pair of tiles, or several CTAs the ranges of one tile's keys.
enum Mode { kWhole = 0, kRange = 1 };

template <int D>
struct Layout {
    static constexpr uint32_t QT = kRows * D * 2;  // one map's queries
    static constexpr uint32_t UT = kKeys * D * 2;  // a unit: 128 keys x d, or 64 keys x 2 d values
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kRing = kQ + 2 * QT;
    static constexpr uint32_t kNorm = kRing + kStages * UT;  // kWhole: [2 D] float, the norm's weights
    // kRange: each row's statistics of both maps, as l = 2^g, [2][kRows] bf16, and m, [2][kRows] float
    static constexpr uint32_t kStatM = kNorm, kStatG = kStatM + 2 * kRows * 4;
    static constexpr uint32_t kBar = kStatG + 2 * kRows * 2;
    // RAW, Q_RAW: FP8 pools' copies complete there; FULL and Q_FULL follow when the rows are f16
    enum { Q_RAW = 0, Q_FULL, Q_FREE, RAW, FULL = RAW + kStages, EMPTY = FULL + kStages,
           ST_FULL = EMPTY + kStages,    // first sweep, per map: scores of a step
           ST_READ = ST_FULL + 2,        // they are in registers
           S2_FULL = ST_READ + 2,        // second sweep: map 2's scores of a step
           S1_FULL = S2_FULL + 1,        // map 1's, per half of the step
           S2_READ = S1_FULL + 2,        // map 2's are in registers
           P_FULL = S2_READ + 1,         // per half: the weights are in tensor memory
           PV_DONE = P_FULL + 2,         // per half: their product has run
           O_FULL = PV_DONE + 2, O_FREE, END_ASK, END_CLEAR, STAT, PARTS, QUAD, DRAIN = QUAD + 4, NBARS };
    static constexpr uint32_t kTmemSlot = kBar + NBARS * 8;
    static constexpr uint32_t kAbort = kTmemSlot + 4;
    static constexpr uint32_t kEnd = kAbort + 4;
    static constexpr size_t bytes = 1024 + kEnd;
    static_assert(bytes <= 232448, "shared memory beyond the 227 KiB a CTA may use");
};

// ------------------------------------------------------------- FP8 pools: E4M3 -> f16 in shared memory

// A tile of R rows x D, converted in place by one warp: rows [row0, row0 + rows).
// Before: E4M3 rows of D bytes in the tile's upper half (the copies' swizzle:
// 16-byte chunk c of row r at c ^ (r & 7) for 128-byte rows, c ^ ((r >> 1) & 3)
// for 64-byte rows).  After: per 64 columns, f16 row r at r * 128 bytes, chunk
// j at j ^ (r & 7).  For D = 128 row r's second 64 columns land exactly on its
// own E4M3 row; for D = 64 f16 row r covers E4M3 rows 2 r - R and 2 r - R + 1,
// none above r (so one warp takes all rows there, in order).  Rows are read
// before any lane writes.
template <int D, int R>
__device__ __forceinline__ void convert_f16(uint32_t tile, int lane, int row0, int rows)
{
    constexpr int CPR = D / 16;      // 16-byte chunks of an E4M3 row
    constexpr int RPI = 32 / CPR;    // rows per step of a warp
    constexpr int U = 4;
    const uint32_t in = tile + R * D;
    const int c = lane % CPR;
#pragma unroll 1
    for (int i = row0; i < row0 + rows; i += U * RPI) {
        uint4 x[U];
        int r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            r[u] = i + u * RPI + lane / CPR;
            const int sw = D == 128 ? r[u] & 7 : (r[u] >> 1) & 3;
            x[u] = lds128(in + r[u] * D + ((c ^ sw) << 4));
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint4 lo, hi;
            e4m3x4_to_f16x4(x[u].x, lo.x, lo.y);
            e4m3x4_to_f16x4(x[u].y, lo.z, lo.w);
            e4m3x4_to_f16x4(x[u].z, hi.x, hi.y);
            e4m3x4_to_f16x4(x[u].w, hi.z, hi.w);
            const uint32_t row = tile + (c >> 2) * (R * 128) + r[u] * 128;
            const int j = 2 * (c & 3);
            sts128(row + ((j ^ (r[u] & 7)) << 4), lo);
            sts128(row + (((j + 1) ^ (r[u] & 7)) << 4), hi);
        }
        __syncwarp();
    }
}

// The tile's queries (bf16, as the copies left them) -> f16 in place, element by element: this warp's share.
template <int D>
__device__ __forceinline__ void convert_q(uint32_t base, int warp, int lane)
{
    constexpr uint32_t share = 2 * Layout<D>::QT / kSoftmaxWarps;
#pragma unroll 4
    for (uint32_t off = warp * share + 16u * lane; off < (warp + 1) * share; off += 16u * 32) {
        uint4 v = lds128(base + off);
        uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = bf16x2_to_f32x2(w[k]);
            w[k] = pack_f16x2(f.x, f.y);
        }
        sts128(base + off, v);
    }
}

// ------------------------------------------------------------- tile walk

struct Tile {
    int b, p, rt0;  // sequence, pair, this CTA's first local row (past R: no rows, it walks along)
    int R;          // rows of (b, p): T * G
    int row0, T, C; // first query token row of b, chunk length, context length (clamped)
    int n_blocks, n_steps;  // blocks the tile sees; steps of this CTA's range
    int s0, S;              // its first step; the tile's steps
};

// A window of 32 sequences or fewer, one per lane: each warp walks the list itself, with the same arithmetic.  The list's
// entries are tiles, sequence by sequence, pair by pair (kRange), or pairs of tiles, within a window those of the
// most steps first (kWhole): dealt out in turns, there and back, they give every cluster close to the same work
// (the 880 entries of 16 prompts of 700 .. 1024 tokens: the longest cluster has 2 % more than the mean, 14 % in the
// order of the sequences).
struct Walker {
    int wb = 0, wbase = 0;           // the window's first sequence, entries before it
    int tot = 0;                     // its entries
    int row0 = 0, T = 0, C = 0;      // this lane's sequence
    int left = 0;                    // its (pairs of) tiles, kWhole: of `steps` steps or fewer
    int incl = 0;                    // entries up to and with this sequence's, kWhole: among those of `steps` steps
    int steps = 0, before = 0;       // kWhole: steps of the entries that are being dealt out; entries of more steps
};

// Steps [range_first(k), range_first(k + 1)) of a tile's S are range k's.
__device__ __forceinline__ int range_first(int S, int ranges, int k) { return (int)((int64_t)S * k / ranges); }

__device__ __forceinline__ int inclusive_sum(int x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// This lane's first pair of tiles with w.steps steps: pair k sees the keys up to C - T + min(T, (k + 1) q).
template <int G>
__device__ __forceinline__ int first_of_class(const Walker &w)
{
    constexpr int q = 2 * kRows / G;  // tokens of a pair of tiles
    const int past = kKeys * (w.steps - 1) - (w.C - w.T);  // of the chunk's tokens, those that fewer steps cover
    return past < 0 ? 0 : past >= w.T ? w.left : min(past / q, w.left);
}

// The entries of the most steps among those left.
template <int G>
__device__ __forceinline__ void next_class(Walker &w, const Args &a, int lane)
{
    constexpr int q = 2 * kRows / G;
    const int seen = w.C - w.T + min(w.T, w.left * q);  // keys of the last pair left
    w.steps = __reduce_max_sync(kFull, w.left > 0 ? (seen + kKeys - 1) / kKeys : 0);
    w.incl = inclusive_sum((w.left - first_of_class<G>(w)) * a.n_pairs, lane);
}

template <int G, int MODE>
__device__ __forceinline__ void load_window(Walker &w, const Args &a, int lane)
{
    const int bl = w.wb + lane;
    w.row0 = w.T = w.C = w.left = 0;
    if (lane < a.window && bl < a.batch) {
        const int32_t lo = a.qo_indptr[bl], hi = a.qo_indptr[bl + 1];
        if (lo < 0 || hi < lo || hi > a.n_rows) {  // rows that are not the caller's: skip the sequence
            atomicOr(a.err, PKV_DEVERR_CTX_RANGE);
        } else {
            w.row0 = lo;
            w.T = hi - lo;
            const int C = a.context_lens[bl], cap = a.W * kBlockSize;
            if (w.T > 0 && (C < w.T || C > cap)) atomicOr(a.err, PKV_DEVERR_CTX_RANGE);
            w.C = max(w.T, min(C, cap));
            constexpr int per = MODE == kWhole ? 2 * kRows : kRows;
            w.left = (w.T * G + per - 1) / per;
        }
    }
    w.incl = inclusive_sum(w.left * a.n_pairs, lane);
    w.tot = __shfl_sync(kFull, w.incl, 31);
    if constexpr (MODE == kWhole) {
        w.before = 0;
        next_class<G>(w, a, lane);
    }
}

// Entry x of the list: CTA `rank`'s tile of the pair, or its range (of `ranges`) of the tile; false past its
// end.  Warp-wide, uniform result.
template <int G, int MODE>
__device__ __forceinline__ bool find_tile(Walker &w, const Args &a, int x, int rank, int ranges, Tile &t, int lane)
{
    while (x >= w.wbase + w.tot) {
        if (w.wb + a.window >= a.batch) return false;
        w.wbase += w.tot;
        w.wb += a.window;
        load_window<G, MODE>(w, a, lane);
    }
    int at = x - w.wbase;
    if constexpr (MODE == kWhole) {
        for (;;) {
            const int tot = __shfl_sync(kFull, w.incl, 31);
            if (at < w.before + tot) break;
            w.before += tot;
            w.left = first_of_class<G>(w);
            next_class<G>(w, a, lane);
        }
        at -= w.before;
    }
    const int l = __ffs(__ballot_sync(kFull, w.incl > at)) - 1;
    const int first = MODE == kWhole ? first_of_class<G>(w) : 0;
    const int nt = __shfl_sync(kFull, w.left - first, l);  // (pairs of) tiles of this sequence among them
    t.b = w.wb + l;
    t.row0 = __shfl_sync(kFull, w.row0, l);
    t.T = __shfl_sync(kFull, w.T, l);
    const int C = __shfl_sync(kFull, w.C, l);
    const int within = at - (__shfl_sync(kFull, w.incl, l) - nt * a.n_pairs);
    t.p = within / nt;
    const int pair0 = (__shfl_sync(kFull, first, l) + within - t.p * nt) * (MODE == kWhole ? 2 : 1) * kRows;
    t.rt0 = pair0 + (MODE == kWhole ? rank * kRows : 0);
    t.s0 = t.S = 0;
    t.R = t.T * G;
    t.C = C;
    if (C > a.W * kBlockSize) {  // a chunk longer than the whole table: nothing sensible to attend to
        t.n_blocks = t.n_steps = 0;
        return true;
    }
    const int last_row = min(t.R, pair0 + (MODE == kWhole ? 2 : 1) * kRows) - 1;  // a pair walks the same keys
    t.n_blocks = (C - t.T + last_row / G) / kBlockSize + 1;
    t.n_steps = (t.n_blocks + kStepBlocks - 1) / kStepBlocks;
    t.S = t.n_steps;
    if constexpr (MODE == kRange) {
        t.s0 = range_first(t.S, ranges, rank);
        t.n_steps = range_first(t.S, ranges, rank + 1) - t.s0;
    }
    return true;
}

// The V unit (of this CTA's 2 n_steps) in which the sequence ends inside a block, or -1.
__device__ __forceinline__ int end_unit(const Tile &t)
{
    if (t.C % kBlockSize == 0 || t.C / kBlockSize >= t.n_blocks) return -1;
    const int v = t.C / kBlockSize / kUnitBlocks - 2 * t.s0;
    return v >= 0 && v < 2 * t.n_steps ? v : -1;
}

// ------------------------------------------------------------- statistics of a row

// (m, l) of both maps, gathered from parts; a part without visible keys has m = -inf, l = 0.
struct RowStat {
    float m1 = -INFINITY, l1 = 0.0f, m2 = -INFINITY, l2 = 0.0f;
    static __device__ __forceinline__ void join(float &m, float &l, float pm, float pl)
    {
        const float top = fmaxf(m, pm);
        const float a = m == -INFINITY ? l : l * ex2(m - top), b = pm == -INFINITY ? pl : pl * ex2(pm - top);
        l = a + b;
        m = top;
    }
    __device__ __forceinline__ void add(float pm1, float pl1, float pm2, float pl2)
    {
        join(m1, l1, pm1, pl1);
        join(m2, l2, pm2, pl2);
    }
    // Weights 2^(s + n0) and 2^(s + n1) of the two maps' scores in log2 units, and o = inv * their sums.
    __device__ __forceinline__ void factors(float abs_lam, float &n0, float &n1, float &inv) const
    {
        if (l1 == 0.0f) {  // a row none of whose blocks could be read stays all zero
            n0 = n1 = inv = 0.0f;
            return;
        }
        // (the approximate forms are off by 2^-21 at most, of what is rounded to 11 bits or fewer; the exact ones
        // take 2 us of 90 where tiles are short.  l1 and l2 are far from 2^126, beyond which __fdividef gives 0.)
        const float c = __fdividef(abs_lam * l1, l2);  // c2 / c1
        n0 = __log2f(c <= 1.0f ? 1.0f : __fdividef(1.0f, c)) + kBoost - m1;
        n1 = __log2f(c <= 1.0f ? c : 1.0f) + kBoost - m2;
        inv = (c <= 1.0f ? __fdividef(1.0f, l1) : __fdividef(abs_lam, l2)) * (1.0f / 256.0f);
    }
};

// Of one map and row (index i), into this CTA's shared memory.  l goes as 2^g with g = log2(l) rounded to bf16
// (there is no room for four floats a row); what the rounding leaves is added to m, so nothing but m's own fp32
// rounding is lost: m + log2(l) is what the weights depend on.
template <typename L>
__device__ __forceinline__ void put_stat(uint8_t *sm, int i, float m, float l)
{
    const float g = log2f(l);
    const __nv_bfloat16 r = __float2bfloat16_rn(m == -INFINITY ? 0.0f : g);
    reinterpret_cast<float *>(sm + L::kStatM)[i] = m == -INFINITY ? m : m + (g - __bfloat162float(r));
    reinterpret_cast<__nv_bfloat16 *>(sm + L::kStatG)[i] = r;
}

// Adds CTA k's of both maps of a row.
template <typename L>
__device__ __forceinline__ void add_stat(RowStat &rs, uint32_t base, int row, int k)
{
    const uint32_t xm = smem_of(base + L::kStatM + row * 4, k), xg = smem_of(base + L::kStatG + row * 2, k);
    const float m1 = ld_cluster_f32(xm), m2 = ld_cluster_f32(xm + 4 * kRows);
    const float g1 = ld_cluster_bf16(xg), g2 = ld_cluster_bf16(xg + 2 * kRows);
    rs.add(m1, m1 == -INFINITY ? 0.0f : ex2(g1), m2, m2 == -INFINITY ? 0.0f : ex2(g2));
}

// ------------------------------------------------------------- the kernel

template <int D, int G, bool F8, int MODE>
__global__ void __launch_bounds__(Warps<F8>::kThreads, 1)
    diff_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                        const __grid_constant__ Args a)
{
    using L = Layout<D>;
    constexpr int NH = D / 64;  // 64-column ranges of a row
    constexpr int NS = L::kStages;
    using Wp = Warps<F8>;
    // FP8 pools: the preparing warps take a quarter of every unit at d_head 128, and half of every other unit at 64
    // (NS is even there, so a warp sees every phase of its slots)
    constexpr int kSplit = !F8 ? 1 : D == 128 ? 4 : 2;  // warps on a unit
    static_assert(Wp::kPreps == kSplit || NS % 2 == 0, "a preparing warp would miss phases of its slots");
    extern __shared__ __align__(1024) uint8_t dp_smem[];
    uint8_t *sm = dp_smem + ((1024u - (smem_u32(dp_smem) & 1023u)) & 1023u);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::kBar);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::kAbort);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);  // the same in all lanes, and known to be
    constexpr bool kPair = MODE == kWhole;
    const int rank = (int)cluster_rank(), ranges = kPair ? 2 : (int)cluster_size();
    // the cluster's entries of the list: there and back in turns (c, 2 N - 1 - c, 2 N + c, ..; kWhole), or one
    const int e0 = (int)(kPair ? blockIdx.x / 2 : blockIdx.x / ranges);
    const int turn = (int)gridDim.x, hop0 = turn - 1 - 2 * e0;  // (2 N)
    const int e_end = kPair ? INT_MAX : e0 + 1;

    if (warp == kCopyWarp && lane == 0) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_kv);
        *abort_flag = 0;
    }
    static_assert(L::NBARS <= 16 * 32, "a thread per barrier");
    {
        const int i = tid;
        if (i < L::NBARS) {
            uint32_t n = 1;
            if (i == L::ST_READ || i == L::ST_READ + 1 || i == L::P_FULL || i == L::P_FULL + 1) n = kSoftmaxWarps / 2;
            if (i == L::S2_READ || i == L::O_FREE) n = kSoftmaxWarps;
            if (i >= L::QUAD && i < L::QUAD + 4) n = 4;  // the four warps of a lane quarter
            if (i == L::Q_FULL && F8) n = kSoftmaxWarps;  // each widens its share of the queries
            if (i >= L::FULL && i < L::EMPTY) n = kSplit;
            if (i == L::STAT) n = 4 * ranges;              // of every CTA, the warps that hold a row's statistics
            if (i == L::PARTS) n = kSoftmaxWarps * ranges;
            if (i == L::DRAIN) n = 2;
            mbar_init(&bar[i], n);
            fence_mbarrier_init();
        }
    }
    if (warp == kScoreWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(sm + L::kTmemSlot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // all CTAs' barriers are ready
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + L::kTmemSlot);
    griddep_wait();
    griddep_launch_dependents();

    auto set_abort = [&]() {
        if (lane == 0) {
            atomicOr(a.err, PKV_DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
    };
    if constexpr (kPair) {
        for (int i = tid; i < 2 * D; i += Wp::kThreads)
            reinterpret_cast<float *>(sm + L::kNorm)[i] = a.w.norm_weight ? a.w.norm_weight[i] : 1.0f;
        __syncthreads();
    }
    Walker wk;
    load_window<G, MODE>(wk, a, lane);
    const uint32_t base = smem_u32(sm);

    if (warp >= kSoftmaxWarps) {
        if constexpr (F8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Wp::kWorkRegs));
        if (warp == kCopyWarp) {
            // ---------------------------------------------------------- copies
            const uint64_t policy = l2_policy_evict_normal();
            int u = 0, n = 0;  // units issued, tiles
            bool ok = true;
            // One lane issues all copies of a unit, the warp running as one: sixteen copies that lanes issued for
            // themselves went out one lane after the other, each moving its operands to uniform registers (1300
            // cycles a unit, which bound the kernel).
            const uint32_t go = elect_one();
            // the next unit: its slot is free, its bytes are announced
            auto open = [&](uint32_t &land, uint32_t &dst) -> bool {
                const int st = u % NS, use = u / NS;
                if (use > 0 && !wait_all(&bar[L::EMPTY + st], (use - 1) & 1)) return false;
                uint64_t *b = &bar[(F8 ? L::RAW : L::FULL) + st];
                land = smem_u32(b);
                dst = base + L::kRing + st * L::UT;
                if (go) mbar_arrive_expect_tx(b, F8 ? L::UT / 2 : L::UT);
                __syncwarp();
                ++u;
                return true;
            };
            for (int x = e0, hop = hop0; ok && x < e_end; x += hop, hop = turn - hop) {
                Tile t;
                if (!find_tile<G, MODE>(wk, a, x, rank, ranges, t, lane)) break;
                if (t.n_steps == 0) continue;
                if (*abort_flag) break;
                if (n > 0 && !(ok = wait_all(&bar[L::Q_FREE], (n - 1) & 1))) break;
                if (lane == 0) {
                    uint64_t *qb = &bar[F8 ? L::Q_RAW : L::Q_FULL];
                    mbar_arrive_expect_tx(qb, 2 * L::QT);
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int h = 0; h < NH; ++h)
                            tma_load_4d(sm + L::kQ + m * L::QT + h * kKHalf, &tm_q, 64 * h, m, t.p * G, t.row0 + t.rt0 / G,
                                        qb, policy);
                }
                ++n;
                const int32_t *trow = a.block_tables + (int64_t)t.b * a.W;
                // lane k < 8: the entry rows of block k's pair of step s, or rows past the pool (zero filled)
                auto rows_of = [&](int s, bool flag) -> int {
                    const int nb = (t.s0 + s) * kStepBlocks + lane;
                    const bool present = lane < kStepBlocks && nb < t.n_blocks;
                    const int id = present ? trow[nb] : -1;
                    const bool valid = id >= 0 && id < a.num_blocks;
                    if (present && !valid && flag) atomicOr(a.err, PKV_DEVERR_BLOCK_RANGE);
                    return valid ? (int)((id * (int64_t)a.n_kv + 2 * t.p) * 2 * kBlockSize) : a.oob_row;
                };
                auto copy_box = [&](uint32_t to, int c, int y, uint32_t land) {
                    tma_load_2d_if(go, to, &tm_kv, c, y, land, policy);
                };
                constexpr int kTileRows = D == 128 ? kKeys : kVKeys;  // of a K unit's tiles, FP8 pools
                auto copy_k = [&](int y0, int m) -> bool {
                    uint32_t land, dst;
                    if (!open(land, dst)) return false;
#pragma unroll
                    for (int k = 0; k < kStepBlocks; ++k) {
                        const int yk = __shfl_sync(kFull, y0, k);
                        const int y = yk == a.oob_row ? yk : yk + m * 2 * kBlockSize;
                        if constexpr (F8) {
                            copy_box(dst + (k * kBlockSize / kTileRows) * (kTileRows * 2 * D) + kTileRows * D +
                                         (k * kBlockSize % kTileRows) * D,
                                     0, y, land);
                        } else {
#pragma unroll
                            for (int h = 0; h < NH; ++h)
                                copy_box(dst + h * kKHalf + k * (kBlockSize * 128), 64 * h, y, land);
                        }
                    }
                    return true;
                };
                auto copy_v = [&](int y0, int h) -> bool {
                    uint32_t land, dst;
                    if (!open(land, dst)) return false;
#pragma unroll
                    for (int k = 0; k < kUnitBlocks; ++k) {
                        const int yk = __shfl_sync(kFull, y0, h * kUnitBlocks + k);
#pragma unroll
                        for (int head = 0; head < 2; ++head) {
                            const int y = yk == a.oob_row ? yk : yk + head * 2 * kBlockSize + kBlockSize;
                            const uint32_t to = dst + head * NH * kVChunk;
                            if constexpr (F8) {
                                copy_box(to + kVKeys * D + k * (kBlockSize * D), 0, y, land);
                            } else {
#pragma unroll
                                for (int c = 0; c < NH; ++c)
                                    copy_box(to + c * kVChunk + k * (kBlockSize * 128), 64 * c, y, land);
                            }
                        }
                    }
                    return true;
                };
                int nxt = rows_of(0, true);
                for (int s = 0; s < t.n_steps && ok; ++s) {
                    const int y0 = nxt;
                    if (s + 1 < t.n_steps) nxt = rows_of(s + 1, true);
                    ok = copy_k(y0, 0) && copy_k(y0, 1);
                }
                if (!ok) break;
                int y0 = rows_of(0, false);
                ok = copy_k(y0, 1) && copy_k(y0, 0);
                for (int s = 0; s < t.n_steps && ok; ++s) {  // in the order of the MMAs
                    if (s + 1 < t.n_steps) nxt = rows_of(s + 1, false);
                    const bool more = s + 1 < t.n_steps;
                    ok = copy_v(y0, 0) && (!more || (copy_k(nxt, 1) && copy_k(nxt, 0))) && copy_v(y0, 1);
                    y0 = nxt;
                }
            }
            // copies still in flight (after an abort) land before the CTA exits
            for (int i = max(0, u - NS); i < u; ++i)
                mbar_wait_bounded(&bar[(F8 ? L::RAW : L::FULL) + i % NS], (i / NS) & 1);
            // and so do the MMAs' arrivals for the last units
            for (int i = max(0, u - NS); i < u && ok && !*abort_flag; ++i)
                ok = wait_all(&bar[L::EMPTY + i % NS], (i / NS) & 1);
            if (n > 0) mbar_wait_bounded(&bar[F8 ? L::Q_RAW : L::Q_FULL], (n - 1) & 1);
            if (!ok) set_abort();
        } else if (warp >= kPrepWarp && warp < Wp::kProduct) {
            // ---------------------------------------------------------- units made ready
            const int which = warp - kPrepWarp;
            {
                int u = 0, ends = 0;
                bool ok = true;
                for (int x = e0, hop = hop0; ok && x < e_end; x += hop, hop = turn - hop) {
                    Tile t;
                    if (!find_tile<G, MODE>(wk, a, x, rank, ranges, t, lane)) break;
                    if (t.n_steps == 0) continue;
                    if (*abort_flag) break;
                    // the V unit the sequence ends inside of: zero the rows behind the end (value heads h0 ..)
                    const int end = end_unit(t), end_row = (t.C / kBlockSize % kUnitBlocks) * kBlockSize;
                    auto clear = [&](uint32_t unit, int h0, int heads) {
                        const int first = end_row + t.C % kBlockSize, rows = end_row + kBlockSize - first;
                        for (int e = lane; e < rows * 8 * heads * NH; e += 32) {
                            const int row = first + (e >> 3) % rows, ch = h0 * NH + (e >> 3) / rows;
                            sts128(unit + ch * kVChunk + row * 128 + (e & 7) * 16, make_uint4(0, 0, 0, 0));
                        }
                    };
                    if constexpr (!F8) {  // the MMA warp asks when the unit has landed
                        if (end >= 0) {
                            const int vs = end / 2, S = t.n_steps;
                            const int v = u + 2 * S + 2 + 4 * vs + (end & 1) * (vs == S - 1 ? 1 : 3);
                            if (!(ok = wait_all(&bar[L::END_ASK], ends & 1))) break;
                            ++ends;
                            clear(base + L::kRing + v % NS * L::UT, 0, 2);
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bar[L::END_CLEAR]);
                        }
                        u += 6 * t.n_steps;
                    } else {
                        for (int i = 0; i < 6 * t.n_steps; ++i, ++u) {
                            const int st = u % NS;
                            if (D == 64 && (u & 1) != which >> 1) continue;
                            if (!(ok = wait_all(&bar[L::RAW + st], (u / NS) & 1))) break;
                            // second sweep: K, K of the first step, then of each step V, K, K, V (the next step's
                            // keys; the last step has V, V)
                            const int iv = i - 2 * t.n_steps - 2;
                            const int vs = iv >> 2, vp = iv & 3;
                            const bool tail = vs == t.n_steps - 1;
                            const bool is_v = iv >= 0 && (tail || vp == 0 || vp == 3);
                            const int vh = vp != 0;  // the V unit's half
                            const uint32_t unit = base + L::kRing + st * L::UT;
                            if constexpr (D == 128) {  // this warp's 32 rows
                                if (is_v) {
                                    const int head = which >> 1, row0 = (which & 1) * 32;
                                    convert_f16<D, kVKeys>(unit + head * NH * kVChunk, lane, row0, 32);
                                    if (2 * vs + vh == end && end_row / 32 == (which & 1)) clear(unit, head, 1);
                                } else {
                                    convert_f16<D, kKeys>(unit, lane, which * 32, 32);
                                }
                            } else {  // half of the keys, or a value head
                                convert_f16<D, kVKeys>(unit + (which & 1) * kVChunk, lane, 0, kVKeys);
                                if (is_v && 2 * vs + vh == end) clear(unit, which & 1, 1);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bar[L::FULL + st]);
                        }
                    }
                }
                if (!ok) set_abort();
            }
        } else if (warp == kScoreWarp || warp == Wp::kProduct) {
            // ---------------------------------------------------------- S_m = Q_m K_m^T and O += W V
            constexpr uint32_t idesc_qk = mma_idesc(kRows, kKeys, 0, F8), idesc_half = mma_idesc(kRows, 64, 0, F8);
            constexpr uint32_t idesc_pv = mma_idesc(kRows, 2 * D, 1, F8);
            const uint64_t qd = smem_desc(base + L::kQ, 16, 1024), kd = smem_desc(base + L::kRing, 16, 1024);
            const uint64_t vd = smem_desc(base + L::kRing, kVChunk, 1024);
            int slot = 0, n = 0;  // of the ring's next unit; tiles
            uint32_t ph = 0;      // the parity of its phase
            int reads = 0, steps = 0, ends = 0;  // first- and second-sweep steps, sequence ends
            const uint32_t go = elect_one();
            const uint32_t tm = __shfl_sync(kFull, tmem, 0);
            auto skip = [&](int k) {
                slot += k;
                if (slot >= NS) {
                    slot -= NS;
                    ph ^= 1u;
                }
            };
            // A slot's barrier has a phase per use.  The two warps wait each for its own units alone, and
            // after what tells it that the slot's use before had been filled: the NS-th unit before is older than
            // those that the weights (or the products) it has just waited for were made from.
            auto unit = [&]() -> bool { return wait_all(&bar[L::FULL + slot], ph); };
            // the unit in slot v has been used when this warp's MMAs so far have run
            auto release = [&](int v) { umma_commit_if(go, &bar[L::EMPTY + v]); };
            // keys [64 half, 64 half + N) of the unit in slot v against map m's queries
            auto scores = [&](int m, int v, int half, uint32_t idesc) {
                tc_fence_after();
                const uint64_t qm = qd + ((m * L::QT) >> 4), km = kd + ((v * L::UT + half * 64 * 128) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * kKHalf + (kk & 3) * 32) >> 4;
                    umma_if(go, tm + m * kKeys + half * 64, qm + off, km + off, idesc, kk > 0 ? 1u : 0u);
                }
            };
            // all of map m's scores of a step
            auto whole = [&](int m, uint64_t *full) -> bool {
                if (!unit()) return false;
                scores(m, slot, 0, idesc_qk);
                umma_commit_if(go, full);
                release(slot);
                skip(1);
                return true;
            };
            auto first_sweep = [&](int s, int m) -> bool {
                // S_m is free: its last scores are in registers, and the weights over S_1 have been used
                if (s > 0) {
                    if (!wait_all(&bar[L::ST_READ + m], (reads - 1) & 1)) return false;
                } else if (n > 0) {
                    if (m == 0 && !(wait_all(&bar[L::PV_DONE], (steps - 1) & 1) && wait_all(&bar[L::PV_DONE + 1], (steps - 1) & 1)))
                        return false;
                    if (m == 1 && !wait_all(&bar[L::S2_READ], (steps - 1) & 1)) return false;
                }
                return whole(m, &bar[L::ST_FULL + m]);
            };
            // map 1's scores of a half, in the second sweep
            auto half_of = [&](int half) {
                scores(0, slot, half, idesc_half);
                umma_commit_if(go, &bar[L::S1_FULL + half]);
                if (half == 1) release(slot);
            };
            auto product = [&](int s, int h, int end) -> bool {
                // (before the unit's wait, see there)
                if (!wait_all(&bar[L::P_FULL + h], steps & 1)) return false;
                if (s == 0 && h == 0 && !wait_all(&bar[L::O_FREE], n & 1)) return false;
                if (!unit()) return false;
                if (!F8 && 2 * s + h == end) {
                    if (go) mbar_arrive(&bar[L::END_ASK]);
                    __syncwarp();
                    if (!wait_all(&bar[L::END_CLEAR], ends & 1)) return false;
                    ++ends;
                }
                tc_fence_after();
                const uint64_t vm = vd + ((slot * L::UT) >> 4);
#pragma unroll
                for (int kk = 0; kk < kVKeys / 16; ++kk)
                    umma_ts_if(go, tm + kColO, tm + h * kVKeys + (kk >> 1) * 32 + (kk & 1) * 8, vm + ((kk * 2048) >> 4), idesc_pv,
                               (s > 0 || h > 0 || kk > 0) ? 1u : 0u);
                umma_commit_if(go, &bar[L::PV_DONE + h]);
                release(slot);
                skip(1);
                return true;
            };
            auto walk = [&](auto on_scores) -> bool {
                constexpr bool kScores = decltype(on_scores)::value;
                for (int x = e0, hop = hop0; x < e_end; x += hop, hop = turn - hop) {
                    Tile t;
                    if (!find_tile<G, MODE>(wk, a, x, rank, ranges, t, lane)) break;
                    if (t.n_steps == 0) continue;
                    if (*abort_flag) break;
                    const int S = __shfl_sync(kFull, t.n_steps, 0);
                    if constexpr (kScores) {
                        if (!wait_all(&bar[L::Q_FULL], n & 1)) return false;
                        for (int s = 0; s < S; ++s, ++reads)
                            if (!(first_sweep(s, 0) && first_sweep(s, 1))) return false;
                        // second sweep: the first step's scores
                        if (!(wait_all(&bar[L::ST_READ + 1], (reads - 1) & 1) && whole(1, &bar[L::S2_FULL]))) return false;
                        if (!(wait_all(&bar[L::ST_READ], (reads - 1) & 1) && unit())) return false;
                        half_of(0);
                        half_of(1);
                        skip(1);
                        for (int s = 0; s + 1 < S; ++s, ++steps) {
                            skip(1);  // V
                            if (!(wait_all(&bar[L::S2_READ], steps & 1) && whole(1, &bar[L::S2_FULL]))) return false;
                            if (!(wait_all(&bar[L::PV_DONE], steps & 1) && unit())) return false;
                            half_of(0);
                            if (!wait_all(&bar[L::PV_DONE + 1], steps & 1)) return false;
                            half_of(1);
                            skip(2);  // and V
                        }
                        umma_commit_if(go, &bar[L::Q_FREE]);
                        ++steps;
                        skip(2);  // V, V
                    } else {
                        const int end = end_unit(t);
                        const int at = (slot + (int)ph * NS + 2 * S + 2) % (2 * NS);  // the first sweep's keys, the first step's
                        slot = at % NS;
                        ph = at >= NS;
                        for (int s = 0; s < S; ++s, ++steps) {
                            if (!product(s, 0, end)) return false;
                            if (s + 1 < S) skip(2);  // keys
                            if (!product(s, 1, end)) return false;
                        }
                        umma_commit_if(go, &bar[L::O_FULL]);
                    }
                    ++n;
                }
                return true;
            };
            bool ok;
            if (warp == kScoreWarp) ok = walk(std::true_type{});
            else ok = walk(std::false_type{});
            umma_commit_if(go, &bar[L::DRAIN]);
            __syncwarp();
            mbar_wait_bounded(&bar[L::DRAIN], 0);
            if (!ok) set_abort();
        }
    } else {
        // ---------------------------------------------------------- statistics, weights, norm
        if constexpr (F8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Wp::kScoreRegs));
        const int quarter = warp & 3, grp = warp >> 2;  // TMEM lanes 32 quarter ..; which of the row's four threads
        const int m = grp & 1, half = grp >> 1;         // first sweep: map, half of a step's keys
        constexpr int QD = D / 2;                       // a thread's channels of the row (of value head grp / 2)
        const int row = quarter * 32 + lane;
        const uint32_t ts = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t to = ts + kColO + grp * QD;
        uint64_t *quad = &bar[L::QUAD + quarter];
        const float lam = diff_lambda<D>(a.w, lane);
        const float abs_lam = fabsf(lam);
        const float sign = lam < 0.0f ? 1.0f : -1.0f;  // of the second map's weights
        const bool rising = a.qscale >= 0.0f;          // the largest score has the largest q . k (else the smallest)
        int gs = 0, ps = 0, n = 0, qph = 0;  // first- and second-sweep steps, tiles, phases of the quad barrier
        bool ok = true;
        // every warp of the quarter is here (and what it wrote to tensor memory is visible)
        auto meet = [&]() -> bool {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(quad);
            const bool done = wait_all(quad, qph & 1);
            ++qph;
            tc_fence_after();
            return done;
        };
        // the next tile that has keys, and this lane's block id of its first step, are found while the tensor
        // cores finish the tile before
        int x = e0, hop = hop0;
        Tile tn;
        int first_id = -1;
        auto find_next = [&]() -> bool {
            do {
                if ((!kPair && x >= e_end) || !find_tile<G, MODE>(wk, a, x, rank, ranges, tn, lane)) return false;
                x += hop;
                hop = turn - hop;
            } while ((kPair ? tn.n_steps : tn.S) == 0);
            const int nb = tn.s0 * kStepBlocks + lane;
            first_id = lane < kStepBlocks && nb < tn.n_blocks ? a.block_tables[(int64_t)tn.b * a.W + nb] : -1;
            return true;
        };
        bool have = find_next();
        while (have && ok) {
            const Tile t = tn;
            const int id0 = first_id;
            if (*abort_flag) break;
            const bool some = kPair || t.n_steps > 0;  // a range may be empty
            if (F8 && some) {
                if (!(ok = wait_all(&bar[L::Q_RAW], n & 1))) break;
                convert_q<D>(base + L::kQ, warp, lane);
                fence_proxy_async_smem();  // the MMAs read it through the async proxy
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[L::Q_FULL]);
            }
            const int r = t.rt0 + row;
            const int pos = t.C - t.T + min(r, t.R - 1) / G;  // this row sees keys 0 .. pos
            const float qs0 = F8 ? a.qscale * a.scales[2 * t.p] : a.qscale;
            const float qs1 = F8 ? a.qscale * a.scales[2 * t.p + 1] : a.qscale;
            const float qs = m == 0 ? qs0 : qs1;
            const int32_t *trow = a.block_tables + (int64_t)t.b * a.W;
            auto ids_of = [&](int s) -> int {
                const int nb = (t.s0 + s) * kStepBlocks + lane;
                return lane < kStepBlocks && nb < t.n_blocks ? trow[nb] : -1;
            };
            // valid blocks of a step, as the copies decided
            auto mask_of = [&](int id) -> uint32_t {
                return __ballot_sync(kFull, lane < kStepBlocks && id >= 0 && id < a.num_blocks);
            };
            // ---- first sweep: maximum and sum of map m over this half's keys ----
            float mx = -INFINITY, l = 0.0f;
            int nxt = id0;
            for (int s = 0; s < t.n_steps; ++s, ++gs) {
                const uint32_t mask = mask_of(nxt) >> (4 * half);
                if (s + 1 < t.n_steps) nxt = ids_of(s + 1);
                if (!(ok = wait_all(&bar[L::ST_FULL + m], gs & 1))) break;
                tc_fence_after();
                uint32_t both[64];
                tmem_ld32(ts + m * kKeys + 64 * half, both);
                tmem_ld32(ts + m * kKeys + 64 * half + 32, both + 32);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[L::ST_READ + m]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {  // 32 keys at a time
                    uint32_t *sr = both + 32 * c;
                    const int key0 = (t.s0 + s) * kKeys + 64 * half + 32 * c;
                    const uint32_t mh = (mask >> (2 * c)) & 3u;
                    if (!__all_sync(kFull, mh == 3u && key0 + 31 <= pos)) {  // what this row does not see never has the largest score
                        const uint32_t never = rising ? 0xff800000u : 0x7f800000u;
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(((mh >> (k / kBlockSize)) & 1u) && key0 + k <= pos)) sr[k] = never;
                    }
                    auto e = [&](int q) { return __uint_as_float(sr[q]); };
                    float mc[4];
                    if (rising) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mc[j] = fmaxf(fmax3(fmax3(fmax3(e(j), e(j + 4), e(j + 8)), e(j + 12), e(j + 16)), e(j + 20), e(j + 24)),
                                          e(j + 28));
                        mc[0] = fmaxf(fmax3(mc[0], mc[1], mc[2]), mc[3]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            mc[j] = e(j);
#pragma unroll
                            for (int q = 1; q < 8; ++q) mc[j] = fminf(mc[j], e(j + 4 * q));
                        }
                        mc[0] = fminf(fminf(mc[0], mc[1]), fminf(mc[2], mc[3]));
                    }
                    const bool none = mc[0] == (rising ? -INFINITY : INFINITY);
                    const float mn = none ? mx : fmaxf(mx, mc[0] * qs);
                    const float neg = mn == -INFINITY ? 0.0f : -mn;
                    float2 sum[4] = {};
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 d = ffma2(make_float2(e(2 * i), e(2 * i + 1)), make_float2(qs, qs), make_float2(neg, neg));
                        sum[i & 3] = fadd2(sum[i & 3], make_float2(ex2(d.x), ex2(d.y)));
                    }
                    const float2 q0 = fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3]));
                    l = (mx == -INFINITY ? 0.0f : l * ex2(mx - mn)) + (q0.x + q0.y);
                    mx = mn;
                }
            }
            if (!ok) break;
            // ---- the row's statistics of both maps give the weights' factors ----
            float n0 = 0.0f, n1 = 0.0f, inv = 0.0f;  // weights 2^(s qs + n); o = inv * accumulator
            RowStat rs;
            if (some) {
                uint32_t st[8] = {__float_as_uint(mx), __float_as_uint(l)};
                tmem_st2(ts + kColStat + 2 * grp, st);
                tmem_wait_st();
                if (!(ok = meet())) break;
                tmem_ld8(ts + kColStat, st);  // (m, l) of threads 0 .. 3: map 1, map 2, map 1, map 2
                tmem_wait_ld();
                auto f = [&](int i) { return __uint_as_float(st[i]); };
                rs.add(f(0), f(1), f(2), f(3));
                rs.add(f(4), f(5), f(6), f(7));
                // O is free: the statistics in its columns, and the tile before, are in registers
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[L::O_FREE]);
            }
            if constexpr (!kPair) {  // every range's
                if (grp == 0) {
                    put_stat<L>(sm, row, rs.m1, rs.l1);
                    put_stat<L>(sm, kRows + row, rs.m2, rs.l2);
                    __syncwarp();
                    if (lane < ranges) mbar_arrive_remote(&bar[L::STAT], lane);
                }
                if (!(ok = wait_all_cluster(&bar[L::STAT], 0))) break;
                rs = RowStat{};
                for (int k = 0; k < ranges; ++k) add_stat<L>(rs, base, row, k);
            }
            rs.factors(abs_lam, n0, n1, inv);
            // ---- second sweep: the weights of keys 32 grp .. + 31 of every step ----
            nxt = id0;
            for (int s = 0; s < t.n_steps; ++s, ++ps) {
                const uint32_t mh = (mask_of(nxt) >> (2 * grp)) & 3u;
                if (s + 1 < t.n_steps) nxt = ids_of(s + 1);
                const int key0 = (t.s0 + s) * kKeys + 32 * grp;
                const bool all = __all_sync(kFull, mh == 3u && key0 + 31 <= pos);
                // map 2's weights first: its scores are there before map 1's, and their place is wanted soonest
                if (!(ok = wait_all(&bar[L::S2_FULL], ps & 1))) break;
                tc_fence_after();
                uint32_t s0[32], s1[32];
                tmem_ld32(ts + kKeys + 32 * grp, s1);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[L::S2_READ]);
                float2 w2[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 u1 = ffma2(make_float2(__uint_as_float(s1[2 * i]), __uint_as_float(s1[2 * i + 1])),
                                            make_float2(qs1, qs1), make_float2(n1, n1));
                    w2[i] = make_float2(ex2(u1.x), ex2(u1.y));
                }
                if (!(ok = wait_all(&bar[L::S1_FULL + half], ps & 1))) break;
                tc_fence_after();
                tmem_ld32(ts + 32 * grp, s0);
                tmem_wait_ld();
                uint32_t pk[16];
                auto weigh = [&](auto masked) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 u0 = ffma2(make_float2(__uint_as_float(s0[2 * i]), __uint_as_float(s0[2 * i + 1])),
                                                make_float2(qs0, qs0), make_float2(n0, n0));
                        float2 w = ffma2(w2[i], make_float2(sign, sign), make_float2(ex2(u0.x), ex2(u0.y)));
                        if constexpr (decltype(masked)::value) {
                            const bool seen = (mh >> (2 * i / kBlockSize)) & 1u;
                            if (!(seen && key0 + 2 * i <= pos)) w.x = 0.0f;
                            if (!(seen && key0 + 2 * i + 1 <= pos)) w.y = 0.0f;
                        }
                        pk[i] = F8 ? pack_f16x2(w.x, w.y) : pack_bf16x2(w.x, w.y);
                    }
                };
                if (all) weigh(std::false_type{});
                else weigh(std::true_type{});
                tmem_st16(ts + 32 * grp, pk);  // over this warp's own scores of map 1, which are read
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[L::P_FULL + half]);
            }
            if (!ok) break;
            // ---- norm and store: this thread's quarter of its row ----
            have = find_next();
            if (some && !(ok = wait_all(&bar[L::O_FULL], n & 1))) break;
            tc_fence_after();
            if constexpr (!kPair) {
                // this range's part of the row into shared memory (the ring's, idle now), 16-byte pieces swizzled
                float4 *part = reinterpret_cast<float4 *>(sm + L::kRing);
                if (some) {
                    const float vs = F8 ? a.scales[a.n_kv + 2 * t.p + half] : 1.0f;
#pragma unroll
                    for (int c = 0; c < QD; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(to + c, o);
                        tmem_wait_ld();
                        if (r < t.R) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int piece = (grp * QD + c) / 4 + i;
                                part[row * (2 * D / 4) + (piece ^ (row & 7))] =
                                    make_float4(__uint_as_float(o[4 * i]) * vs, __uint_as_float(o[4 * i + 1]) * vs,
                                                __uint_as_float(o[4 * i + 2]) * vs, __uint_as_float(o[4 * i + 3]) * vs);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane < ranges) mbar_arrive_remote(&bar[L::PARTS], lane);
                if (!(ok = wait_all_cluster(&bar[L::PARTS], 0))) break;
                // rows rank, rank + ranges, ...: a warp adds the ranges' parts in order, normalises and stores
                const int live = min(kRows, t.R - t.rt0);
                for (int q = rank + warp * ranges; q < live; q += kSoftmaxWarps * ranges) {
                    constexpr int KW = 2 * D / 128;
                    float4 o[KW];
#pragma unroll
                    for (int c = 0; c < KW; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
                    RowStat all;
                    for (int k = 0; k < ranges; ++k) {
                        add_stat<L>(all, base, q, k);
                        if (range_first(t.S, ranges, k) == range_first(t.S, ranges, k + 1)) continue;  // no steps
#pragma unroll
                        for (int c = 0; c < KW; ++c) {
                            const int piece = lane + 32 * c;
                            const float4 y = ld_cluster_f32x4(
                                smem_of(base + L::kRing + (q * (2 * D / 4) + (piece ^ (q & 7))) * 16, k));
                            o[c].x += y.x;
                            o[c].y += y.y;
                            o[c].z += y.z;
                            o[c].w += y.w;
                        }
                    }
                    float x0, x1, fac;
                    all.factors(abs_lam, x0, x1, fac);
                    float ss = 0.0f;
#pragma unroll
                    for (int c = 0; c < KW; ++c) {
                        o[c].x *= fac;
                        o[c].y *= fac;
                        o[c].z *= fac;
                        o[c].w *= fac;
                        ss += o[c].x * o[c].x + o[c].y * o[c].y + o[c].z * o[c].z + o[c].w * o[c].w;
                    }
#pragma unroll
                    for (int s = 16; s >= 1; s >>= 1) ss += __shfl_xor_sync(kFull, ss, s);
                    const float rn = a.w.out_scale * rsqrtf(ss * (1.0f / (2 * D)) + a.w.eps);
                    const int rq = t.rt0 + q;
                    __nv_bfloat16 *dst = a.out + (((int64_t)t.row0 + rq / G) * (a.n_q / 2) + t.p * G + rq % G) * (2 * D);
#pragma unroll
                    for (int c = 0; c < KW; ++c) {
                        const int d = 4 * (lane + 32 * c);
                        const float4 g = a.w.norm_weight ? __ldg(reinterpret_cast<const float4 *>(a.w.norm_weight + d))
                                                         : make_float4(1.f, 1.f, 1.f, 1.f);
                        *reinterpret_cast<uint2 *>(dst + d) = make_uint2(pack_bf16x2(o[c].x * rn * g.x, o[c].y * rn * g.y),
                                                                         pack_bf16x2(o[c].z * rn * g.z, o[c].w * rn * g.w));
                    }
                }
                break;
            }
            const float f = inv * (F8 ? a.scales[a.n_kv + 2 * t.p + half] : 1.0f);
            uint32_t o[QD];
#pragma unroll
            for (int c = 0; c < QD; c += 32) tmem_ld32(to + c, o + c);
            tmem_wait_ld();
            float2 sq[2] = {};
#pragma unroll
            for (int i = 0; i < QD / 2; ++i) {
                const float2 v = make_float2(__uint_as_float(o[2 * i]) * f, __uint_as_float(o[2 * i + 1]) * f);
                o[2 * i] = __float_as_uint(v.x);
                o[2 * i + 1] = __float_as_uint(v.y);
                sq[i & 1] = ffma2(v, v, sq[i & 1]);
            }
            float ss = (sq[0].x + sq[0].y) + (sq[1].x + sq[1].y);
            {
                uint32_t z = __float_as_uint(ss);
                tmem_st1(to, z);  // this thread's part of O is in registers
                tmem_wait_st();
                if (!(ok = meet())) break;
                uint32_t y[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) tmem_ld1(ts + kColO + g * QD, y[g]);
                tmem_wait_ld();
                ss = (__uint_as_float(y[0]) + __uint_as_float(y[1])) + (__uint_as_float(y[2]) + __uint_as_float(y[3]));
            }
            const float rn = a.w.out_scale * rsqrtf(ss * (1.0f / (2 * D)) + a.w.eps);
            // The row's pieces of 32 bytes change places among the lanes of NP rows, so that a store instruction
            // writes whole pieces of 32 / NP rows instead of 32: the load-store unit passes once for each row that
            // an instruction touches (9 of 355 us).
            constexpr int NP = QD / 16;
            uint32_t w[NP][8];
            const float4 *nw = reinterpret_cast<const float4 *>(sm + L::kNorm) + grp * (QD / 4);
#pragma unroll
            for (int c = 0; c < NP; ++c) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 g = nw[4 * c + i];
                    const uint32_t *x4 = o + 16 * c + 4 * i;
                    w[c][2 * i] = pack_bf16x2(__uint_as_float(x4[0]) * rn * g.x, __uint_as_float(x4[1]) * rn * g.y);
                    w[c][2 * i + 1] = pack_bf16x2(__uint_as_float(x4[2]) * rn * g.z, __uint_as_float(x4[3]) * rn * g.w);
                }
            }
#pragma unroll
            for (int d = NP / 2; d >= 1; d >>= 1) {  // piece c of lane l and piece c ^ d of lane l ^ d
                const bool up = lane & d;
#pragma unroll
                for (int c = 0; c < NP; ++c) {
                    if (c & d) continue;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t y = __shfl_xor_sync(kFull, up ? w[c][i] : w[c + d][i], d);
                        if (up) w[c][i] = y;
                        else w[c + d][i] = y;
                    }
                }
            }
            // now w[c] is piece `lane % NP` of the row of lane (lane - lane % NP + c)
#pragma unroll
            for (int c = 0; c < NP; ++c) {
                const int rc = t.rt0 + quarter * 32 + (lane & ~(NP - 1)) + c;
                if (rc < t.R)
                    stg256(a.out + (((int64_t)t.row0 + rc / G) * (a.n_q / 2) + t.p * G + rc % G) * (2 * D) + grp * QD +
                               16 * (lane & (NP - 1)),
                           w[c]);
            }
            ++n;
        }
        if (!ok) set_abort();
    }

    tc_fence_before();
    __syncthreads();  // every role is done with the tensor memory
    cluster_sync();   // the others' last commits, copies and reads of this CTA's shared memory are done
    tc_fence_after();
    if (warp == kScoreWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ------------------------------------------------------------- launch

// A launch of clusters of `size` CTAs.
template <int D, int G, bool F8, int MODE>
struct ClusterLaunch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    ClusterLaunch(int clusters, int size, cudaStream_t s)
    {
        cfg.gridDim = dim3(clusters * size);
        cfg.blockDim = dim3(Warps<F8>::kThreads);
        cfg.dynamicSmemBytes = Layout<D>::bytes;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = size;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
    }
};

// Per device, found once: the kernel's attributes are set, and resident[i] clusters of 2^(i + 1) CTAs are
// resident at once (kRange).
template <int D, int G, bool F8, int MODE>
pkv_status prepare(const pkv_pool *pool, int (&resident)[4])
{
    struct Known {
        bool ready;
        int resident[4];
    };
    static std::mutex mu;
    static Known known[64];
    std::lock_guard<std::mutex> lock(mu);
    Known local = {}, *k = pool->device < 64 ? &known[pool->device] : &local;
    if (!k->ready) {
        auto kern = diff_prefill_kernel<D, G, F8, MODE>;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::bytes);
        if (e == cudaSuccess && MODE == kRange) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        cudaFuncAttributes fa;
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kern);
        if (e != cudaSuccess) return cuda_fail(e, "paged_diff_prefill_attention: kernel attributes");
        // (with fewer registers at the launch, the warps on scores would wait for theirs)
        if (F8 && fa.numRegs < Warps<F8>::kLaunchRegs)
            return fail(PKV_EUNSUPPORTED, "paged_diff_prefill_attention: built with %d registers a thread", fa.numRegs);
        for (int i = 0; i < 4 && MODE == kRange; ++i) {
            ClusterLaunch<D, G, F8, MODE> cl(1, 2 << i, nullptr);
            cl.cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&k->resident[i], kern, &cl.cfg) != cudaSuccess) {
                cudaGetLastError();  // a size the device does not take
                k->resident[i] = 0;
            }
        }
        k->ready = true;
    }
    for (int i = 0; i < 4; ++i) resident[i] = k->resident[i];
    return PKV_OK;
}

template <int D, int G, bool F8, int MODE>
pkv_status launch_mode(pkv_pool *pool, const CUtensorMap &tm_q, int clusters, int size, const Args &a, cudaStream_t s)
{
    ClusterLaunch<D, G, F8, MODE> cl(clusters, size, s);
    LaunchScope ls(pool, kDecode, s);
    cudaError_t e = cudaLaunchKernelEx(&cl.cfg, diff_prefill_kernel<D, G, F8, MODE>, tm_q, pool->tm_block, a);
    ls.done();
    if (e != cudaSuccess) return cuda_fail(e, "paged_diff_prefill_attention launch");
    return PKV_OK;
}

// The most tiles of `per` rows that n_rows tokens of `batch` sequences can make: each sequence that has rows one,
// and one for every `per` rows beyond its first row (sum of 1 + floor((x_i - 1) / per) over x_i > 0).
int64_t most_tiles(int64_t n_rows, int G, int batch, int per)
{
    const int64_t begun = std::min<int64_t>(batch, n_rows);
    return begun + (n_rows * G - begun) / per;
}

template <int D, int G, bool F8>
pkv_status launch(pkv_pool *pool, const void *q, Args a, cudaStream_t s)
{
    CUtensorMap tm_q;
    pkv_status st = make_q_pair_map(&tm_q, q, a.n_rows, a.n_q, D, G, kRows / G);
    if (st != PKV_OK) return st;
    const int64_t tiles = most_tiles(a.n_rows, G, a.batch, kRows) * a.n_pairs;
    const int64_t pairs = most_tiles(a.n_rows, G, a.batch, 2 * kRows) * a.n_pairs;
    const int64_t steps = (a.W + kStepBlocks - 1) / kStepBlocks;  // of the longest sequence the table can hold
    int resident[4];
    a.window = 32;
    // ranges: the largest cluster of which all tiles' (counting the most the call can have) run at once
    if (tiles <= pool->num_sms / 2 && steps > 1) {
        st = prepare<D, G, F8, kRange>(pool, resident);
        if (st != PKV_OK) return st;
        for (int i = 3; i >= 0; --i)
            if (tiles <= resident[i] && (2 << i) <= std::max<int64_t>(2, steps))
                return launch_mode<D, G, F8, kRange>(pool, tm_q, (int)tiles, 2 << i, a, s);
    }
    st = prepare<D, G, F8, kWhole>(pool, resident);
    if (st != PKV_OK) return st;
    // Windows of few sequences keep what runs together within the L2, those of many entries even out the clusters'
    // work: four entries a cluster (16 prompts of 700 .. 1024 tokens: 357 us with 8 sequences, 370 with 16; 24 of
    // 129 .. 1023 at d_head 64: 103 with 8, 91 with 16, 93 with 32).
    const int clusters = (int)std::min<int64_t>(pairs, pool->num_sms / 2);
    for (a.window = 4; a.window < 32 && pairs * a.window < (int64_t)4 * clusters * a.batch;) a.window *= 2;
    return launch_mode<D, G, F8, kWhole>(pool, tm_q, clusters, 2, a, s);
}

template <int D, bool F8>
pkv_status dispatch_g(pkv_pool *pool, const void *q, int G, const Args &a, cudaStream_t s)
{
    switch (G) {
    case 1: return launch<D, 1, F8>(pool, q, a, s);
    case 2: return launch<D, 2, F8>(pool, q, a, s);
    case 4: return launch<D, 4, F8>(pool, q, a, s);
    case 8: return launch<D, 8, F8>(pool, q, a, s);
    }
    return fail(PKV_EUNSUPPORTED, "differential prefill: group size %d unsupported (1, 2, 4 or 8)", G);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status paged_diff_prefill_attention(pkv_pool *pool, const void *q, int64_t n_rows, int32_t n_q,
                                                   const int32_t *qo_indptr, const int32_t *block_tables,
                                                   int32_t max_blocks_per_seq, const int32_t *context_lens,
                                                   int32_t batch, float scale, const pkv_diff_params *params, void *out,
                                                   void *stream)
{
    const char *who = "paged_diff_prefill_attention";
    pkv_status st = check_step_args(pool, who, n_q, max_blocks_per_seq, batch, scale);
    Args a;
    if (st == PKV_OK) st = check_diff_args(pool, who, params, &a.w);
    if (st != PKV_OK) return st;
    if (n_rows < 0) return fail(PKV_EINVAL, "%s: n_rows < 0", who);
    if (batch == 0 || n_rows == 0) return PKV_OK;
    const int G = n_q / pool->n_kv;
    if (n_rows > INT32_MAX / G) return fail(PKV_EUNSUPPORTED, "%s: more than 2^31 query rows x group size", who);
    if (!q || !qo_indptr || !block_tables || !context_lens || !out)
        return fail(PKV_EINVAL, "%s: NULL device pointer", who);
    if (((uintptr_t)q & 15u) || ((uintptr_t)out & 31u))
        return fail(PKV_EINVAL, "%s: q must be 16-byte and out 32-byte aligned", who);
    if (((uintptr_t)qo_indptr | (uintptr_t)block_tables | (uintptr_t)context_lens) & 3u)
        return fail(PKV_EINVAL, "%s: indptr, tables and lengths must be 4-byte aligned", who);
    st = check_pool_device(pool, who);
    if (st != PKV_OK) return st;
    if (most_tiles(n_rows, G, batch, kRows) * (pool->n_kv / 2) > INT32_MAX) return fail(PKV_EUNSUPPORTED, "%s: too many query rows", who);
    a.qo_indptr = qo_indptr;
    a.block_tables = block_tables;
    a.W = max_blocks_per_seq;
    a.context_lens = context_lens;
    a.batch = batch;
    a.n_q = n_q;
    a.n_kv = pool->n_kv;
    a.n_pairs = pool->n_kv / 2;
    a.num_blocks = pool->num_blocks;
    a.n_rows = n_rows;
    a.oob_row = (int)(pool->num_blocks * pool->n_kv * 2 * kBlockSize);
    // (0 as 1e-30: the same scores to fp32, but -inf for hidden ones stays -inf)
    a.qscale = scale == 0.0f ? 1e-30f : scale * kLog2e;
    a.scales = pool->scales;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.err = pool->err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f8 = pool->dtype == PKV_FP8_E4M3;
    if (pool->d_head == 128)
        return f8 ? dispatch_g<128, true>(pool, q, G, a, s) : dispatch_g<128, false>(pool, q, G, a, s);
    return f8 ? dispatch_g<64, true>(pool, q, G, a, s) : dispatch_g<64, false>(pool, q, G, a, s);
}
