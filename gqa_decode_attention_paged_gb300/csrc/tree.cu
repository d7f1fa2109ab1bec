// Attention of a tree of drafted tokens over the paged cache, on the tcgen05
// tensor cores.
//
// Mathematics.  Node i of sequence b (row qo_indptr[b] + i) sits at cached
// position C - T + i; for query head h of KV head g
//   out = sum_p softmax_p(s q_ih . K_pg) V_pg
// over the positions before the nodes and the nodes j whose bit is set in row
// i's mask.  The rows of one KV head are (node i, head h of its group), row
// i * G + h.  One pass over the keys with a running maximum and sum; a key
// that a row does not see has score -infinity.
//
// What bounds it: HBM, while a KV head's rows are few (up to 256 of them read the
// cache once, 4 d rows operations for every 4 d bytes of a bf16 key and value),
// the tensor cores and the exponentials from about 256 rows on.  Every further
// 256 rows of a KV head read the cache again: they follow one another in the
// stream, and the L2 has little left of what the first ones read (64 nodes on
// 16 x 8192 tokens, 512 rows a KV head: 1087 MB from HBM for 531 MB of cache).
//
// Design (one persistent CTA per SM, warp-specialised):
//   * a unit is up to 256 rows (two tiles of 128) of one (sequence, KV head).
//     The stream of all units' steps of 128 keys, weighed by what they cost, is
//     cut into one equal slice per CTA, so that every SM has the same work
//     whatever the lengths are, and one long sequence keeps all of them busy (64
//     trees of 1..60 nodes on an E4M3 cache: 201 us with all steps weighed
//     alike, 149 so).  A unit that a slice holds whole is finished by its CTA; of
//     one that is cut each CTA leaves its part (reference maximum, sum,
//     unnormalised O), which tree_merge_kernel joins.  A slice cuts at most two
//     units, the one it starts inside of (partial slot 2 cta) and the one it ends
//     inside of (2 cta + 1).  Where units are small, or there is one per SM and
//     they are about alike, none is cut (see kCostCut).
//   * two streams of softmax, each with its own scores and accumulator in
//     tensor memory and its own eight warps: while one forms weights, the tensor
//     cores work for the other.  A unit of two tiles gives each stream a tile,
//     and both use every key and value tile; in a unit of one tile the streams
//     take alternate steps (the second one the first, as it is the first that
//     joins the two by log-sum-exp at the end).
//   * a softmax warp has 16 rows, all 64 keys of a turn, read from tensor
//     memory as a matrix product's result is laid out: four threads a row, which
//     two shuffles reduce.  (A thread per row, four warps a stream, left every
//     scheduler with two warps and their dependent chains.)
//   * one warp walks the slice, says what the next piece of work is (a queue of
//     four in shared memory: where every warp walked for itself, the softmax
//     warps spilled), and streams what the MMAs take through one ring of 32 KiB
//     (d 128) tiles: keys of a step, its values, keys of the next.  Two warps issue one stream's MMAs
//     each: S = Q K^T, and when the weights are written over S, O += P V.
//   * the reference maximum is raised lazily (O is rescaled only when a row's
//     maximum grows by more than 2^8).  Weights are rounded to bf16 (FP8 pools:
//     f16, times 2^7) for the MMA; the sum adds them in fp32 as they were (adding the
//     rounded ones takes twice the additions, and makes no measurable difference
//     against 64 bits).
//   * FP8 pools: the E4M3 tiles are widened to f16 in place by four warps.
//   * value rows behind the sequence's end are zeroed in shared memory before
//     their product: a weight of 0 does not cancel what is not finite.  Nodes that
//     a row does not see may hold anything, too: what is not finite in the nodes'
//     value rows becomes 0 there, and is added to the results of the rows that see
//     it, whatever their scores, when the slice is done (16 trees of 17..32 nodes on 1024..2048 tokens: 38 us
//     without the look at the nodes' rows, 39 with it).
// Every mbarrier wait is bounded; on a timeout the CTA records
// PKV_DEVERR_TIMEOUT, every role stops, the MMA and copy pipes are drained
// (bounded) and the tensor memory is released before the CTA exits.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <mutex>

#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kRows = 128;                 // query rows per tile (= TMEM lanes)
constexpr int kUnitRows = 2 * kRows;
constexpr int kKeys = 128;                 // keys per step
constexpr int kStepBlocks = kKeys / kBlockSize;
constexpr int kTurn = 64;                  // keys that a softmax warp takes at a time
constexpr int kTurnBlocks = kTurn / kBlockSize;
constexpr int kSoftmaxWarps = 16;
constexpr int kCopyWarp = 16, kMmaWarp = 17, kPrepWarp = 20;
constexpr int kMaxWords = 16;
constexpr int kMany = 4;                   // windows of 32 sequences whose lengths are read at a time
// What a step costs in a unit of one tile (bound by HBM, or by the widening of its keys) and of two (by the products
// and exponentials), and a unit besides its steps: about 1.4, 2 and 4 us.  (16 trees of 17..32 nodes on 1024..2048 tokens
// and 64 of 1..60 on E4M3: 38.1 and 131 us so, 38.8 and 140 with 3, 4 and 6, 38.9 and 128..135 with units at half more.)
constexpr int kCostOne = 2, kCostTwo = 3, kCostUnit = 6;
constexpr int kMinShare = kCostUnit + 2 * kCostOne;  // of a slice
// (between two steps' beginnings: no slice inside a unit is without one)
static_assert(kMinShare >= kCostUnit + kCostTwo, "");
// Units are not cut where that would gain less than it costs (a second beginning and end, the parts, the join).  With 16
// nodes on four heads, 8 KV heads, us a call, cut and whole:
//   * no more units than CTAs, one each: where the costliest is above the even share by kCostCut at most.  128 units on
//     1024, 2048, 4096 tokens: 28.3 / 19.7, 37.7 / 32.2, 53.7 / 52.2; 64 units on 1536 (18 above): 23.2 / 23.5; on 2048
//     (23 above): 25.4 / 28.0; 8 on 1024 (21 above): 15.9 / 17.5.
//   * more units than CTAs, to the slice in which they begin: where none costs more than kCostSmall.  512 units on 1024,
//     1536, 2048 tokens (22, 30, 38): 73 / 65, 85.7 / 84.2, 99.9 / 102.9; 1024 units on 1536: 152 / 156.
constexpr int kCostCut = 18, kCostSmall = 30;
// And where tables have no more steps than this, so that the join need not be launched: with tables of 1024 tokens 8, 32,
// 512 units take 15.9 / 15.9, 20.0 / 16.3, 73 / 66; with 1536, 15.2 / 20.1, 20.5 / 20.1, 86 / 86.  (The table's width decides,
// as the host does not see the lengths: 8 nodes on 300 tokens take 8.7 us in a graph with a table of 19 blocks, 9.0 with 64,
// 10.0 with 65 and 10.3 with 2048.)
constexpr int kWholeSteps = 8;
template <bool F8>
struct Warps {
    static constexpr int kWarps = F8 ? 24 : 20, kThreads = kWarps * 32;
    // registers a thread at the launch, then of the softmax warps and of the others
    static constexpr int kLaunchRegs = F8 ? 80 : 96, kScoreRegs = F8 ? 96 : 104, kWorkRegs = F8 ? 48 : 64;
    static_assert(kSoftmaxWarps * kScoreRegs + (kWarps - kSoftmaxWarps) * kWorkRegs <= kWarps * kLaunchRegs,
                  "more registers than the launch has");
};
// Tensor memory: S_x at 128 x, two places of 64 columns (fp32 scores of a turn; its weights, packed in pairs, over the
// first 32), O_x at 256 + D x.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;
constexpr uint32_t kHalf = 128 * 128;      // bytes of a 64-column range of a 128-row tile
constexpr float kSlack = 8.0f;             // log2 of the largest weight before the reference maximum is raised
// FP8 pools: log2 of a factor of all weights, which their sum has too.  f16 ends at 2^16, and loses bits below 2^-14: so
// what weighs down to 2^-21 of the reference is held to 2^-11 of itself (2^-14 without; of many keys that weighed 2^-25
// of the first one, nothing was left).
constexpr float kLift = 7.0f;
static_assert(kSlack + kLift < 16.0f, "weights beyond f16's range");

// The unit that a CTA's slice has a part of and that goes on in the next one, for the merge.  more < 0: none.
struct Part {
    int row0, r0, R, g;  // first token row, first local row, local rows, KV head
    int more, back;      // parts that follow the first; which of them this CTA's is
};

struct Args {
    const int32_t *qo_indptr;  // [batch + 1]
    const uint32_t *mask;      // [n_rows][2 words]
    int words;
    const int32_t *block_tables;
    int W;
    const int32_t *context_lens;
    int batch, n_q, n_kv;
    const uint8_t *pool;
    int64_t num_blocks, n_rows;
    int oob_row;          // a row index past the end of the pool's entry rows (zero-filled box)
    float qscale;         // scale * log2(e)
    const float *scales;  // FP8 pools: [2 * n_kv] fp32, K scales then V scales
    bool whole;           // no unit is cut, whatever they cost
    int slot_rows;        // rows of a partial slot
    Part *parts;          // [CTAs]
    float2 *ws_ml;        // [2 CTAs][slot_rows] (reference maximum in log2 units, sum)
    float *ws_o;          // [2 CTAs][slot_rows][D] unnormalised
    __nv_bfloat16 *out;   // [n_rows][n_q][D]
    unsigned *err;
};

template <int D>
struct Layout {
    static constexpr uint32_t QT = kRows * D * 2;  // a tile of queries
    static constexpr uint32_t UT = kKeys * D * 2;  // a step's keys, or its values
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kRing = kQ + 2 * QT;
    static constexpr uint32_t kStat = kRing + kStages * UT;  // a unit of one tile: stream 1's (m, l) per row
    static constexpr int kQueue = 4;
    static constexpr uint32_t kPieces = kStat + kRows * 8;   // what to do next, 64 bytes each
    static constexpr uint32_t kBar = kPieces + kQueue * 64;
    // RAW, Q_RAW: FP8 pools' copies complete there; FULL and Q_FULL follow when the rows are f16
    enum { Q_RAW = 0, Q_FULL, Q_FREE, RAW, FULL = RAW + kStages, EMPTY = FULL + kStages,
           S_FULL = EMPTY + kStages,  // per stream and place: scores of a turn
           P_FULL = S_FULL + 4,       // its weights are in tensor memory
           PV_DONE = P_FULL + 4,      // their product has run
           STAT = PV_DONE + 4,        // per warp of a stream: stream 1's statistics and O are final
           TAKEN = STAT + 8,          // they are read
           NEXT = TAKEN + 8,          // a piece of the queue is there
           DONE = NEXT + kQueue,      // every warp is done with it
           DRAIN = DONE + kQueue, NBARS };
    static constexpr uint32_t kTmemSlot = kBar + NBARS * 8;
    static constexpr uint32_t kAbort = kTmemSlot + 4;
    static constexpr uint32_t kOdd = kAbort + 4;    // a value of a node was not finite
    static constexpr uint32_t kSlice = kOdd + 4;    // where the CTA's slice begins
    static constexpr uint32_t kEnd = kSlice + 28;
    static constexpr size_t bytes = 1024 + kEnd;
    static_assert(bytes <= 232448, "shared memory beyond the 227 KiB a CTA may use");
};

// A tile of R rows x D E4M3 -> f16, in place, by one warp: rows [row0, row0 + rows).
// Before: rows of D bytes in the tile's upper half (the copies' swizzle: 16-byte
// chunk c of row r at c ^ (r & 7) for 128-byte rows, c ^ ((r >> 1) & 3) for
// 64-byte rows).  After: per 64 columns, f16 row r at r * 128 bytes, chunk j at
// j ^ (r & 7).  For D = 128 row r's second 64 columns land exactly on its own
// E4M3 row; for D = 64 f16 row r covers E4M3 rows 2 r - R and 2 r - R + 1, none
// above r (so one warp takes all rows there, in order).  Rows are read before any
// lane writes.
template <int D, int R>
__device__ __forceinline__ void widen(uint32_t tile, int lane, int row0, int rows)
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

// What is not finite in rows [r0, r1) of a tile becomes 0, and *odd 1 before that (a second warp that does the same
// and finds the 0 finds the 1, too).
template <int D, bool F8>
__device__ __forceinline__ void zero_odd(uint32_t tile, int lane, int r0, int r1, volatile int *odd)
{
    constexpr int NH = D / 64;
    constexpr uint32_t kExp = F8 ? 0x7c007c00u : 0x7f807f80u, kUp = F8 ? 0x04000400u : 0x00800080u;
#pragma unroll 4
    for (int e = r0 * 8 * NH + lane; e < r1 * 8 * NH; e += 32) {
        const uint32_t at = tile + (e >> 3) % NH * kHalf + (e >> 3) / NH * 128 + (e & 7) * 16;
        uint4 v = lds128(at);
        // an exponent of ones carries into the sign's place
        auto bad = [&](uint32_t w) { return ((w & kExp) + kUp) & 0x80008000u; };
        if (bad(v.x) | bad(v.y) | bad(v.z) | bad(v.w)) {
            *odd = 1;
            __threadfence_block();
            auto clear = [&](uint32_t w) { return w & ~((bad(w) >> 15) * 0xffffu); };
            sts128(at, make_uint4(clear(v.x), clear(v.y), clear(v.z), clear(v.w)));
        }
    }
}

// ------------------------------------------------------------- the stream of steps

// Steps [s0, s0 + n) of a unit: what a CTA does of it.
struct Piece {
    int b, g, r0;      // sequence, KV head, first local row
    int row0, T, R, C; // first token row, nodes, local rows (nodes x heads), cache length
    int S, s0, n;      // the unit's steps; this piece's
    int more, back;    // pieces of the unit in the slices that follow, and in those before
    int next;          // where the stream goes on
    int blocks;        // of the sequence
    // the first of the piece's steps that has nodes, and the rows of a step's tile that are nodes
    __device__ __forceinline__ int node_step() const { return (C - T) / kKeys - s0; }
    __device__ __forceinline__ int node0(int s) const { return max(0, C - T - (s0 + s) * kKeys); }
    __device__ __forceinline__ int node1(int s) const { return min(kKeys, C - (s0 + s) * kKeys); }
    __device__ __forceinline__ bool two() const { return R - r0 > kRows; }
    __device__ __forceinline__ bool whole() const { return n == S; }
};

// A window of 32 sequences, one per lane.
struct Walker {
    int wb = 0, wbase = 0, tot = 0;  // first sequence of the window, costs before it, its costs
    int incl = 0;                    // costs up to and with this lane's sequence
    int row0 = 0, T = 0, C = 0;      // this lane's sequence
    int units = 0, most = 0;         // of the lane's sequences so far: units, and the cost of the costliest
    bool whole = false;              // units belong to the slice in which they begin
    bool index = false;              // and count one each
};

__device__ __forceinline__ int inclusive_sum(int x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// The units of a sequence and KV head with R rows and S steps: all but the last have two tiles.  In a unit of step cost
// w, step 0 begins at 0 and step s at kCostUnit + w s.
struct Units {
    int n, full, last;  // units, size of all but the last in the stream, of the last
    int step;           // step cost of the last
    int all;            // size of the whole
    __device__ __forceinline__ Units(int R, int S, bool index)
    {
        n = (R + kUnitRows - 1) / kUnitRows;
        step = R - (n - 1) * kUnitRows > kRows ? kCostTwo : kCostOne;
        full = index ? 1 : S * kCostTwo + kCostUnit;
        last = index ? 1 : S * step + kCostUnit;
        all = (n - 1) * full + last;
    }
    // steps that begin before x
    static __device__ __forceinline__ int begun(int x, int w)
    {
        return x <= 0 ? 0 : max(1, (x - kCostUnit + w - 1) / w);
    }
};

// Sequence b's nodes and length; its size in the stream, none where it does not fit.
template <int G>
__device__ __forceinline__ int sequence(const Args &a, int b, Walker &w, bool flag)
{
    w.row0 = w.T = w.C = 0;
    if (b >= a.batch) return 0;
    const int lo = a.qo_indptr[b], hi = a.qo_indptr[b + 1], C = a.context_lens[b];
    if (lo < 0 || hi < lo || hi > a.n_rows || hi - lo > 64 * a.words || C < hi - lo || C > a.W * kBlockSize) {
        if (flag) atomicOr(a.err, PKV_DEVERR_CTX_RANGE);
        return 0;
    }
    if (hi == lo) return 0;
    w.row0 = lo;
    w.T = hi - lo;
    w.C = C;
    const Units u(w.T * G, (C + kKeys - 1) / kKeys, w.index);
    w.units += u.n * a.n_kv;
    w.most = max(w.most, u.n > 1 ? u.full : u.last);
    return u.all * a.n_kv;
}

template <int G>
__device__ __forceinline__ void load_window(Walker &w, const Args &a, int lane, bool flag)
{
    const int work = sequence<G>(a, w.wb + lane, w, flag);
    w.incl = inclusive_sum(work, lane);
    w.tot = __shfl_sync(kFull, w.incl, 31);
}

// The piece that begins at f in the stream, up to `end`; false past it.  A step belongs to the slice in which it
// begins.  Warp-wide, uniform result.
template <int G>
__device__ __forceinline__ bool find_piece(Walker &w, const Args &a, int f, int end, int share, Piece &p, int lane)
{
    for (;;) {
        if (f >= end) return false;
        while (f >= w.wbase + w.tot) {
            if (w.wb + 32 >= a.batch) return false;
            w.wbase += w.tot;
            w.wb += 32;
            load_window<G>(w, a, lane, false);
        }
        const int at = f - w.wbase;
        const int l = __ffs(__ballot_sync(kFull, w.incl > at)) - 1;
        p.b = w.wb + l;
        p.row0 = __shfl_sync(kFull, w.row0, l);
        p.T = __shfl_sync(kFull, w.T, l);
        p.C = __shfl_sync(kFull, w.C, l);
        p.S = (p.C + kKeys - 1) / kKeys;
        p.R = p.T * G;
        const Units u(p.R, p.S, w.index);
        const int within = at - (__shfl_sync(kFull, w.incl, l) - u.all * a.n_kv);
        p.g = within / u.all;
        int x = within - p.g * u.all;  // in the KV head, then in the unit
        const int unit = min(x / u.full, u.n - 1);
        x -= unit * u.full;
        p.r0 = unit * kUnitRows;
        const int size = unit == u.n - 1 ? u.last : u.full;
        if (w.whole) {
            if (x > 0) {  // the slice before has it
                f += size - x;
                continue;
            }
            p.s0 = p.more = p.back = 0;
            p.n = p.S;
            p.next = f + size;
        } else {
            const int cost = unit == u.n - 1 ? u.step : kCostTwo, e = min(size, x + (end - f));
            p.s0 = Units::begun(x, cost);
            p.n = (e == size ? p.S : Units::begun(e, cost)) - p.s0;
            p.next = f + (e - x);
            // the last step's beginning, behind this slice's end
            const int left = (p.S == 1 ? 0 : kCostUnit + cost * (p.S - 1)) - e;
            p.more = left < 0 ? 0 : left / share + 1;
            p.back = f / share - (f - x) / share;
        }
        p.blocks = (p.C + kBlockSize - 1) / kBlockSize;
        if (p.n > 0) return true;
        f = p.next;
    }
}

// Bits [at, at + 32) of a row's view of its sequence's T nodes; the positions before the nodes are all seen.
__device__ __forceinline__ uint32_t node_bits(const uint32_t *row, int words, int T, int at)
{
    if (at <= -32) return kFull;
    if (at >= T) return 0;
    auto word = [&](int i) -> uint32_t { return i >= 0 && i < words ? __ldg(row + i) : i < 0 ? kFull : 0u; };
    const int i = at >> 5;  // (rounds down: -1 where the 32 begin before the nodes)
    uint32_t bits = __funnelshift_r(word(i), word(i + 1), at & 31);
    if (T - at < 32) bits &= (1u << (T - at)) - 1u;
    return bits;
}

// Adds what zero_odd took out of a piece's nodes to the rows [t0, t0 + 16) that see it, as this warp has stored them:
// in out, or unnormalised at `part`.
template <int D, int G, bool F8>
__device__ __forceinline__ void add_odd(const Args &a, const Piece &p, int t0, float *part, int lane)
{
    constexpr int PL = D / 32;  // channels of a lane
    constexpr int KV = F8 ? PKV_FP8_E4M3 : PKV_BF16;
    constexpr int64_t ROWB = kv_row_bytes(KV, D), ENTRY = kv_entry_bytes(KV, D);
    const int at0 = p.C - p.T, j1 = min(p.T, (p.s0 + p.n) * kKeys - at0);
#pragma unroll 1
    for (int j = max(0, p.s0 * kKeys - at0); j < j1; ++j) {
        const int pos = at0 + j, id = a.block_tables[(int64_t)p.b * a.W + pos / kBlockSize];
        if (id < 0 || id >= a.num_blocks) continue;
        const uint8_t *v = a.pool + ((int64_t)id * a.n_kv + p.g) * ENTRY + kv_v_offset(KV, D) + pos % kBlockSize * ROWB;
        float x[PL];
        bool odd = false;
#pragma unroll
        for (int d = 0; d < PL; ++d) {
            const int c = lane * PL + d;
            if constexpr (F8) x[d] = (v[c] & 0x7f) == 0x7f ? NAN : 0.0f;
            else x[d] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(v)[c]);
            if (x[d] - x[d] == 0.0f) x[d] = 0.0f;  // (finite)
            else odd = true;
        }
        if (!__any_sync(kFull, odd)) continue;
#pragma unroll 1
        for (int r = t0; r < min(t0 + 16, p.R); ++r) {
            const int64_t row = (int64_t)p.row0 + r / G;
            if (!((a.mask[row * 2 * a.words + (j >> 5)] >> (j & 31)) & 1u)) continue;
            __nv_bfloat16 *dst = a.out + (row * a.n_q + p.g * G + r % G) * D;
#pragma unroll
            for (int d = 0; d < PL; ++d) {
                const int c = lane * PL + d;
                if (x[d] == 0.0f) continue;
                if (part) part[(int64_t)(r - p.r0) * D + c] += x[d];
                else dst[c] = __float2bfloat16(__bfloat162float(dst[c]) + x[d]);
            }
        }
    }
}

// Where a CTA's slice begins and ends, and in which window of 32 sequences.
struct Slice {
    int f0, f1, share, wb, wbase, whole, index;
};

// The same for all rows that a softmax warp (w8 of stream x) has stored.
template <int D, int G, bool F8>
__device__ __noinline__ void add_odd_rows(const Args &a, const Slice &from, int x, int t0, int lane)
{
    Walker wk;
    wk.wb = from.wb;
    wk.wbase = from.wbase;
    wk.whole = from.whole;
    wk.index = from.index;
    load_window<G>(wk, a, lane, false);
    Piece p;
    for (int f = from.f0; find_piece<G>(wk, a, f, from.f1, from.share, p, lane); f = p.next) {
        if (!p.two() && x == 1) continue;
        float *part = p.whole() ? nullptr : a.ws_o + (2 * (int64_t)blockIdx.x + (p.s0 == 0 ? 1 : 0)) * a.slot_rows * D;
        add_odd<D, G, F8>(a, p, p.r0 + (p.two() ? x * kRows : 0) + t0, part, lane);
    }
}

// ------------------------------------------------------------- the kernel

template <int D, int G, bool F8>
__global__ void __launch_bounds__(Warps<F8>::kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                const __grid_constant__ Args a)
{
    using L = Layout<D>;
    using Wp = Warps<F8>;
    constexpr int NH = D / 64;  // 64-column ranges of a row
    constexpr int NS = L::kStages;
    constexpr int kWarps = Wp::kThreads / 32;
    // FP8 pools: the preparing warps take a quarter of every tile at d_head 128, and half of every other tile at 64
    // (NS is even there, so a warp sees every phase of its slots)
    constexpr int kSplit = !F8 ? 1 : D == 128 ? 4 : 2;  // warps on a tile
    static_assert(D == 128 || NS % 2 == 0, "a preparing warp would miss phases of its slots");
    extern __shared__ __align__(1024) uint8_t tree_smem[];
    uint8_t *sm = tree_smem + ((1024u - (smem_u32(tree_smem) & 1023u)) & 1023u);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::kBar);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::kAbort);
    volatile int *odd_flag = reinterpret_cast<volatile int *>(sm + L::kOdd);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);  // the same in all lanes, and known to be

    if (warp == kCopyWarp && lane == 0) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_kv);
        *abort_flag = *odd_flag = 0;
    }
    static_assert(L::NBARS <= Wp::kThreads, "a thread per barrier");
    if (tid < L::NBARS) {
        const int i = tid;
        uint32_t n = 1;
        if (i >= L::P_FULL && i < L::P_FULL + 4) n = kSoftmaxWarps / 2;  // a stream's warps
        if (i == L::Q_FREE || i == L::DRAIN) n = 2;                // both issuing warps
        if (i >= L::EMPTY && i < L::EMPTY + NS) n = 2;
        if (i >= L::DONE && i < L::DONE + L::kQueue) n = kSoftmaxWarps + 2 + (F8 ? 4 : 0);
        if (i == L::Q_FULL && F8) n = 4;                           // the preparing warps widen the queries
        if (i >= L::FULL && i < L::FULL + NS) n = kSplit;
        mbar_init(&bar[i], n);
        fence_mbarrier_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(sm + L::kTmemSlot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
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

    const uint32_t base = smem_u32(sm);
    // The queue's piece i, when it is there (n == 0: no more; null: time ran out); and the warp is done with it.
    auto next_piece = [&](int i) -> const Piece * {
        if (*abort_flag || !wait_all(&bar[L::NEXT + i % L::kQueue], (i / L::kQueue) & 1)) return nullptr;
        return reinterpret_cast<const Piece *>(sm + L::kPieces + i % L::kQueue * 64);
    };
    auto done_with = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[L::DONE + i % L::kQueue]);
    };

    if (warp >= kCopyWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Wp::kWorkRegs));
        if (warp == kCopyWarp) {
            // ---------------------------------------------------------- copies
            // ---- this CTA's slice of the stream, and the window in which it begins ----
            Walker wk;
            int total = 0, many0 = 0, many1 = 0, f0, f1, share;
            static_assert(kMaxBatch <= 64 * 32 * kMany, "");
            auto scan = [&](bool flag) {
                total = 0;
                if (a.batch <= 32) {
                    load_window<G>(wk, a, lane, flag);
                    total = wk.tot;
                    return;
                }
                for (int b = 0; b < a.batch; b += 32 * kMany) {
                    int x = 0;
#pragma unroll
                    for (int i = 0; i < kMany; ++i) x += sequence<G>(a, b + 32 * i + lane, wk, flag);
                    x = __reduce_add_sync(kFull, x);
                    total += x;
                    const int i = b / (32 * kMany);  // lane i % 32 keeps it
                    if (lane == i % 32) (i < 32 ? many0 : many1) = x;
                }
            };
            scan(blockIdx.x == 0);
            share = (total + (int)gridDim.x - 1) / (int)gridDim.x;
            const int units = __reduce_add_sync(kFull, wk.units), most = __reduce_max_sync(kFull, wk.most);
            wk.index = units <= (int)gridDim.x && (a.whole || most <= share + kCostCut);
            wk.whole = wk.index || a.whole || (units > (int)gridDim.x && most <= kCostSmall);
            share = max(share, kMinShare);
            if (wk.index) {
                scan(false);
                share = 1;
            }
            f0 = min((int64_t)total, (int64_t)blockIdx.x * share);
            f1 = min((int64_t)total, (int64_t)f0 + share);
            if (a.batch > 32) {
                const int incl0 = inclusive_sum(many0, lane), all0 = __shfl_sync(kFull, incl0, 31), incl1 = all0 + inclusive_sum(many1, lane);
                const unsigned on0 = __ballot_sync(kFull, incl0 - many0 <= f0), on1 = __ballot_sync(kFull, incl1 - many1 <= f0);
                // the last that begins at or before f0 (those behind the batch begin at its end)
                const int i = on1 ? 63 - __clz(on1) : 31 - __clz(on0);
                wk.wb = min(i * 32 * kMany, a.batch - 1) / (32 * kMany) * (32 * kMany);
                const int j = wk.wb / (32 * kMany);
                wk.wbase = __shfl_sync(kFull, j < 32 ? incl0 - many0 : incl1 - many1, j % 32);
                load_window<G>(wk, a, lane, false);
            }
            if (lane == 0) *reinterpret_cast<Slice *>(sm + L::kSlice) = {f0, f1, share, wk.wb, wk.wbase, wk.whole, wk.index};
            const uint64_t policy = l2_policy_evict_normal();
            const uint32_t go = elect_one();  // one lane issues all copies, the warp running as one
            int u = 0, n = 0;                 // tiles of the ring, pieces
            bool ok = true;
            Part cut = {0, 0, 0, 0, -1, 0};
            for (int f = f0;;) {
                if (*abort_flag) break;
                Piece p;
                const bool some = find_piece<G>(wk, a, f, f1, share, p, lane);
                if (!some) p.n = 0;
                const int slot = n % L::kQueue;
                if (n >= L::kQueue && !(ok = wait_all(&bar[L::DONE + slot], (n / L::kQueue - 1) & 1))) break;
                if (lane == 0) {
                    *reinterpret_cast<Piece *>(sm + L::kPieces + slot * 64) = p;
                    mbar_arrive(&bar[L::NEXT + slot]);
                }
                __syncwarp();
                if (!some) break;
                f = p.next;
                // The queries go out behind the first step's tiles: those need no more than what the piece before
                // leaves of the ring, the queries that it has issued its last scores.
                auto copy_q = [&]() -> bool {
                    if (n > 0 && !wait_all(&bar[L::Q_FREE], (n - 1) & 1)) return false;
                    if (lane == 0) {
                        uint64_t *qb = &bar[F8 ? L::Q_RAW : L::Q_FULL];
                        mbar_arrive_expect_tx(qb, p.two() ? 2 * L::QT : L::QT);
                        for (int t = 0; t < (p.two() ? 2 : 1); ++t)
#pragma unroll
                            for (int h = 0; h < NH; ++h)
                                tma_load_3d(sm + L::kQ + t * L::QT + h * kHalf, &tm_q, 64 * h, p.g * G,
                                            p.row0 + (p.r0 + t * kRows) / G, qb, policy);
                    }
                    __syncwarp();
                    return true;
                };
                static_assert(NS >= 2, "");
                if (p.more > 0) cut = {p.row0, p.r0, p.R, p.g, p.back + p.more, p.back};
                const int32_t *trow = a.block_tables + (int64_t)p.b * a.W;
                // lane k < 8: the entry rows of block k of a step, or rows past the pool (zero filled)
                auto rows_of = [&](int s) -> int {
                    const int nb = (p.s0 + s) * kStepBlocks + lane;
                    const bool present = lane < kStepBlocks && nb < p.blocks;
                    const int id = present ? trow[nb] : -1;
                    const bool valid = id >= 0 && id < a.num_blocks;
                    if (present && !valid) atomicOr(a.err, PKV_DEVERR_BLOCK_RANGE);
                    return valid ? (int)((id * (int64_t)a.n_kv + p.g) * 2 * kBlockSize) : a.oob_row;
                };
                int nxt = rows_of(0);
                for (int s = 0; s < p.n && ok; ++s) {
                    const int y0 = nxt;
                    if (s + 1 < p.n) nxt = rows_of(s + 1);
#pragma unroll
                    for (int v = 0; v < 2; ++v, ++u) {  // keys, then values
                        const int st = u % NS, use = u / NS;
                        if (use > 0 && !(ok = wait_all(&bar[L::EMPTY + st], (use - 1) & 1))) break;
                        uint64_t *b = &bar[(F8 ? L::RAW : L::FULL) + st];
                        const uint32_t land = smem_u32(b), dst = base + L::kRing + st * L::UT;
                        if (go) mbar_arrive_expect_tx(b, F8 ? L::UT / 2 : L::UT);
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < kStepBlocks; ++k) {
                            const int yk = __shfl_sync(kFull, y0, k);
                            const int y = yk == a.oob_row ? yk : yk + v * kBlockSize;
                            if constexpr (F8) {
                                constexpr int kTileRows = D == 128 ? 128 : 64;  // (see widen)
                                tma_load_2d_if(go, dst + (k * kBlockSize / kTileRows) * (kTileRows * 2 * D) + kTileRows * D +
                                                       (k * kBlockSize % kTileRows) * D,
                                               &tm_kv, 0, y, land, policy);
                            } else {
#pragma unroll
                                for (int h = 0; h < NH; ++h)
                                    tma_load_2d_if(go, dst + h * kHalf + k * (kBlockSize * 128), &tm_kv, 64 * h, y, land, policy);
                            }
                        }
                    }
                    if (ok && s == 0) ok = copy_q();
                }
                if (!ok) break;
                ++n;
            }
            if (lane == 0) a.parts[blockIdx.x] = cut;
            // copies still in flight (after an abort) land before the CTA exits
            for (int i = max(0, u - NS); i < u; ++i)
                mbar_wait_bounded(&bar[(F8 ? L::RAW : L::FULL) + i % NS], (i / NS) & 1);
            // and so do the MMAs' arrivals for the last tiles
            for (int i = max(0, u - NS); i < u && ok && !*abort_flag; ++i)
                ok = wait_all(&bar[L::EMPTY + i % NS], (i / NS) & 1);
            for (int i = max(0, n - 1); i <= n && !ok; ++i) mbar_wait_bounded(&bar[F8 ? L::Q_RAW : L::Q_FULL], i & 1, kWaitLimitNs / 4);
            if (n > 0 && ok) ok = wait_all(&bar[F8 ? L::Q_RAW : L::Q_FULL], (n - 1) & 1);
            if (!ok) set_abort();
        } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            // ---------------------------------------------------------- S = Q K^T and O += P V of one stream
            // A turn is 64 keys.  A stream's scores have two places, so that the next turn's are there when the
            // softmax has written this one's weights.
            const int x = warp - kMmaWarp;
            constexpr uint32_t idesc_qk = mma_idesc(kRows, kTurn, 0, F8), idesc_pv = mma_idesc(kRows, D, 1, F8);
            const uint32_t tm = __shfl_sync(kFull, tmem, 0);
            const uint32_t go = elect_one();
            const uint64_t kd = smem_desc(base + L::kRing, 16, 1024), vd = smem_desc(base + L::kRing, kHalf, 1024);
            int u0 = 0, n = 0, turns = 0;  // tiles of the ring and turns of this stream before the piece; pieces
            bool ok = true;
            auto full = [&](int i) -> bool { return wait_all(&bar[L::FULL + i % NS], (i / NS) & 1); };
            auto landed = [&](int i) -> bool { return __all_sync(kFull, mbar_test(&bar[L::FULL + i % NS], (i / NS) & 1)); };
            for (;;) {
                const Piece *pp = next_piece(n);
                if (!(ok = pp != nullptr)) break;
                const Piece &p = *pp;
                if (p.n == 0) break;
                // (the same in all lanes, and known to be: an MMA whose operands are not takes 80 cycles to issue)
                const bool two = __shfl_sync(kFull, (int)p.two(), 0);
                const int steps = __shfl_sync(kFull, p.n, 0), nodes = __shfl_sync(kFull, p.node_step(), 0);
                const bool tail = !F8 && p.s0 + steps == p.S && p.C % kBlockSize;
                const int hop = two ? 1 : 2, s1 = two ? 0 : 1 - x;        // this stream's steps: s1, s1 + hop, ..
                const int last = 2 * ((steps - s1 + hop - 1) / hop);      // its turns
                const uint64_t qd = smem_desc(base + L::kQ + (two ? x * L::QT : 0), 16, 1024);
                if (!(ok = wait_all(&bar[L::Q_FULL], n & 1))) break;
                int passed = two ? steps : 0;  // the other stream's steps before it have been passed
                // of the other stream's steps before s: only say that their tiles are not needed here (any more)
                auto pass = [&](int s) -> bool {
                    for (; passed < s; ++passed) {
                        if ((passed & 1) != x) continue;
                        const int u = u0 + 2 * passed;
                        if (!full(u) || !full(u + 1)) return false;
                        if (go) {
                            mbar_arrive(&bar[L::EMPTY + u % NS]);
                            mbar_arrive(&bar[L::EMPTY + (u + 1) % NS]);
                        }
                        __syncwarp();
                    }
                    return true;
                };
                auto scores = [&](int t) -> bool {
                    const int s = s1 + (t >> 1) * hop, half = t & 1, u = u0 + 2 * s, st = u % NS, at = (turns + t) & 1;
                    if (half == 0 && !(pass(s) && full(u))) return false;
                    // the place is free: the weights over its last scores, two turns ago, have been used
                    if (turns + t >= 2 && !wait_all(&bar[L::PV_DONE + 2 * x + at], ((turns + t - 2) >> 1) & 1)) return false;
                    tc_fence_after();
                    const uint64_t km = kd + ((st * L::UT + half * kTurn * 128) >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                        umma_if(go, tm + x * kKeys + at * kTurn, qd + off, km + off, idesc_qk, kk > 0 ? 1u : 0u);
                    }
                    umma_commit_if(go, &bar[L::S_FULL + 2 * x + at]);
                    if (half) umma_commit_if(go, &bar[L::EMPTY + st]);
                    if (t == last - 1) umma_commit_if(go, &bar[L::Q_FREE]);
                    return true;
                };
                auto product = [&](int t) -> bool {
                    const int s = s1 + (t >> 1) * hop, half = t & 1, u = u0 + 2 * s + 1, st = u % NS, at = (turns + t) & 1;
                    if (half == 0) {
                        if (!full(u)) return false;
                        if (tail && s == steps - 1) {
                            // the sequence ends inside a block: zero the value rows behind its end (both streams of
                            // two tiles do, each before its own product; the second writes zeros over zeros)
                            const int r0 = p.C % kKeys, rows = kBlockSize - p.C % kBlockSize;
                            for (int e = lane; e < rows * 8 * NH; e += 32) {
                                const int row = r0 + (e >> 3) % rows, h = (e >> 3) / rows;
                                sts128(base + L::kRing + st * L::UT + h * kHalf + row * 128 + (e & 7) * 16, make_uint4(0, 0, 0, 0));
                            }
                        }
                        if (!F8 && s >= nodes) zero_odd<D, F8>(base + L::kRing + st * L::UT, lane, p.node0(s), p.node1(s), odd_flag);
                        if (!F8 && (s >= nodes || (tail && s == steps - 1))) {
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                    if (!wait_all(&bar[L::P_FULL + 2 * x + at], ((turns + t) >> 1) & 1)) return false;
                    tc_fence_after();
                    const uint64_t vm = vd + ((st * L::UT + half * kTurn * 128) >> 4);
#pragma unroll
                    for (int kk = 0; kk < kTurn / 16; ++kk)
                        umma_ts_if(go, tm + kColO + x * D, tm + x * kKeys + at * kTurn + kk * 8, vm + ((kk * 2048) >> 4), idesc_pv,
                                   t > 0 || kk > 0 ? 1u : 0u);
                    umma_commit_if(go, &bar[L::PV_DONE + 2 * x + at]);
                    if (half) umma_commit_if(go, &bar[L::EMPTY + st]);
                    return true;
                };
                if (last == 0) umma_commit_if(go, &bar[L::Q_FREE]);  // (a piece of one step has none for stream 0)
                else ok = scores(0);
                for (int t = 0; t < last && ok; ++t) {
                    // the next turn's scores first, unless their keys have not come yet: values wait for nothing then
                    const int u = u0 + 2 * (s1 + ((t + 1) >> 1) * hop);
                    const bool more = t + 1 < last;
                    const bool early = more && ((t + 1) & 1 || (landed(u) && (two || (landed(u - 1) && landed(u - 2)))));
                    if (early && !(ok = scores(t + 1))) break;
                    if (!(ok = product(t))) break;
                    if (more && !early) ok = scores(t + 1);
                }
                if (ok) ok = pass(steps);
                if (!ok) break;
                u0 += 2 * steps;
                turns += last;
                done_with(n);
                ++n;
            }
            umma_commit_if(go, &bar[L::DRAIN]);
            __syncwarp();
            mbar_wait_bounded(&bar[L::DRAIN], 0);
            if (!ok) set_abort();
        } else if (F8 && warp >= kPrepWarp && warp < kPrepWarp + 4) {
            // ---------------------------------------------------------- E4M3 tiles widened
            const int which = warp - kPrepWarp;
            int u = 0;  // tiles of the ring
            bool ok = true;
            // the queries to f16 in place, element by element: this warp's quarter
            auto widen_q = [&](int n, bool two) -> bool {
                if (!wait_all(&bar[L::Q_RAW], n & 1)) return false;
                const uint32_t part = (two ? 2 : 1) * L::QT / 4;
#pragma unroll 4
                for (uint32_t off = which * part + 16u * lane; off < (which + 1) * part; off += 16u * 32) {
                    uint4 v = lds128(base + off);
                    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 q = bf16x2_to_f32x2(w[k]);
                        w[k] = pack_f16x2(q.x, q.y);
                    }
                    sts128(base + off, v);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[L::Q_FULL]);
                return true;
            };
            for (int n = 0;; ++n) {  // pieces
                const Piece *pp = next_piece(n);
                if (!(ok = pp != nullptr)) break;
                const Piece &p = *pp;
                if (p.n == 0) break;
                const int nodes = p.node_step();
                for (int i = 0; i < 2 * p.n; ++i, ++u) {
                    // (the first keys are widened before the queries, which come when the piece before is done with its own)
                    if (i == 1 && !(ok = widen_q(n, p.two()))) break;
                    if (D == 64 && (u & 1) != which >> 1) continue;
                    const int st = u % NS;
                    if (!(ok = wait_all(&bar[L::RAW + st], (u / NS) & 1))) break;
                    const uint32_t tile = base + L::kRing + st * L::UT;
                    constexpr int kOwn = D == 128 ? 32 : 64;  // rows of this warp
                    const int own0 = D == 128 ? which * 32 : (which & 1) * 64;
                    if constexpr (D == 128) widen<D, 128>(tile, lane, own0, 32);
                    else widen<D, 64>(tile + own0 * 128, lane, 0, 64);
                    if ((i & 1) && p.s0 + (i >> 1) == p.S - 1 && p.C % kBlockSize) {  // value rows behind the end
                        const int r0 = p.C % kKeys, rows = kBlockSize - p.C % kBlockSize;
                        if (r0 / kOwn * kOwn == own0) {
                            for (int e = lane; e < rows * 8 * NH; e += 32) {
                                const int row = r0 + (e >> 3) % rows, h = (e >> 3) / rows;
                                sts128(tile + h * kHalf + row * 128 + (e & 7) * 16, make_uint4(0, 0, 0, 0));
                            }
                        }
                    }
                    if ((i & 1) && (i >> 1) >= nodes)  // (the rows are written: widen ends with a warp's barrier)
                        zero_odd<D, F8>(tile, lane, max(p.node0(i >> 1), own0), min(p.node1(i >> 1), own0 + kOwn), odd_flag);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[L::FULL + st]);
                }
                if (!ok) break;
                done_with(n);
            }
            if (!ok) set_abort();
        }
    } else {
        // ---------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Wp::kScoreRegs));
        const int x = warp >> 3, w8 = warp & 7;            // stream, warp of it
        const int row0 = (w8 & 3) * 32 + (w8 >> 2) * 16;   // its rows (TMEM lanes) row0 .. + 15
        const int g8 = lane >> 2, c4 = lane & 3;           // this thread's rows row0 + g8, + 8; its pair of every 8 columns
        const uint32_t ts = tmem + ((uint32_t)row0 << 16);
        float2 *stat = reinterpret_cast<float2 *>(sm + L::kStat);
        const bool rising = a.qscale >= 0.0f;  // else scores are negated as they are read
        int turns = 0, joins = 0;              // this stream's turns, units of one tile
        bool ok = true;
        for (int i = 0; ok; ++i) {  // pieces
            const Piece *pp = next_piece(i);
            if (!(ok = pp != nullptr)) break;
            const Piece &p = *pp;
            const int n = p.n;
            if (n == 0) break;
            const bool two = p.two();
            const int t0 = p.r0 + (two ? x * kRows : 0) + row0;  // the warp's first local row
            const bool live = t0 < p.R;
            const int rel0 = p.s0 * kKeys - (p.C - p.T);         // the first step's first key, against the first node
            // (never 0, which times a hidden key's -inf would be NaN: a product below fp32's range is its least normal number)
            const float qs = F8 ? fmaxf(fabsf(a.qscale) * a.scales[p.g], FLT_MIN) : fabsf(a.qscale), vs = F8 ? a.scales[a.n_kv + p.g] : 1.0f;
            const int32_t *trow = a.block_tables + (int64_t)p.b * a.W + p.s0 * kStepBlocks;
            const int blocks = p.blocks - p.s0 * kStepBlocks;
            const int hop = two ? 1 : 2, s1 = two ? 0 : 1 - x;
            auto node = [&](int i) -> int { return min(t0 + g8 + 8 * i, p.R - 1) / G; };  // of this thread's row i
            auto ids_of = [&](int s) -> int {
                return lane < kStepBlocks && s < n && s * kStepBlocks + lane < blocks ? trow[s * kStepBlocks + lane] : -1;
            };
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};  // of the rows; sums of this thread's keys
            int nxt = ids_of(s1);
            uint32_t valid = 0;
            for (int s = s1, t = 0; s < n; s += hop * (t & 1), ++t, ++turns) {  // (two turns a step)
                const int half = t & 1;
                if (half == 0) {  // blocks that are there, as the copies decided
                    valid = __ballot_sync(kFull, lane < kStepBlocks && nxt >= 0 && nxt < a.num_blocks);
                    nxt = ids_of(s + hop);
                }
                const uint32_t place = ts + x * kKeys + (turns & 1) * kTurn;
                if (!(ok = wait_all(&bar[L::S_FULL + 2 * x + (turns & 1)], (turns >> 1) & 1))) break;
                if (live) {
                    tc_fence_after();
                    uint32_t pk[kTurn / 4];  // words 2 n + i: row i's weights of keys 8 n + 2 c4, + 1
                    float add[2], alpha[2] = {1.0f, 1.0f};
                    // Weights are formed with the reference as it is, while the maximum is found; the rare turn that
                    // raises it reads the scores again.  (A piece's first one finds the maximum first.)
                    bool fresh = t == 0, again = false;
                    do {
                        uint32_t sr[kTurn / 2];  // words 4 n + 2 i + e: row i's key 8 n + 2 c4 + e
                        tmem_ld_rows64(place, sr);
                        tmem_wait_ld();
                        if (!rising) {
#pragma unroll
                            for (int i = 0; i < kTurn / 2; ++i) sr[i] ^= 0x80000000u;
                        }
                        const int rel = rel0 + s * kKeys + half * kTurn;
                        const uint32_t there = (valid >> (half * kTurnBlocks)) & ((1u << kTurnBlocks) - 1);
                        if (rel + kTurn > 0 || there != (1u << kTurnBlocks) - 1) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t *mrow = a.mask + ((int64_t)p.row0 + node(i)) * 2 * a.words;
#pragma unroll
                                for (int c = 0; c < kTurn / 32; ++c) {
                                    uint32_t bits = node_bits(mrow, 2 * a.words, p.T, rel + 32 * c);
                                    if (!((there >> (2 * c)) & 1u)) bits &= 0xffff0000u;
                                    if (!((there >> (2 * c)) & 2u)) bits &= 0xffffu;
                                    bits >>= 2 * c4;
#pragma unroll
                                    for (int k = 0; k < 8; ++k)
                                        if (!((bits >> (8 * (k >> 1) + (k & 1))) & 1u)) sr[16 * c + 4 * (k >> 1) + 2 * i + (k & 1)] = 0xff800000u;
                                }
                            }
                        }
                        auto e = [&](int i, int k) { return __uint_as_float(sr[4 * (k >> 1) + 2 * i + (k & 1)]); };  // row i's k-th key here
                        float top[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float mx[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) mx[j] = fmaxf(fmax3(e(i, j), e(i, j + 4), e(i, j + 8)), e(i, j + 12));
                            top[i] = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
                        }
                        auto reduce = [&]() {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                top[i] = fmaxf(top[i], __shfl_xor_sync(kFull, top[i], 1));
                                top[i] = fmaxf(top[i], __shfl_xor_sync(kFull, top[i], 2)) * qs;
                            }
                        };
                        if (fresh) {
                            reduce();
                            m[0] = top[0];
                            m[1] = top[1];
                        }
                        constexpr float lift = F8 ? kLift : 0.0f;
                        const float nm[2] = {m[0] == -INFINITY ? 0.0f : lift - m[0], m[1] == -INFINITY ? 0.0f : lift - m[1]};
                        float2 part[2][2] = {};
#pragma unroll
                        for (int j = 0; j < kTurn / 8; ++j) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float2 d = ffma2(make_float2(e(i, 2 * j), e(i, 2 * j + 1)), make_float2(qs, qs), make_float2(nm[i], nm[i]));
                                const float2 w = make_float2(ex2(d.x), ex2(d.y));
                                part[i][j & 1] = fadd2(part[i][j & 1], w);
                                pk[2 * j + i] = F8 ? pack_f16x2(w.x, w.y) : pack_bf16x2(w.x, w.y);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 y = fadd2(part[i][0], part[i][1]);
                            add[i] = y.x + y.y;
                        }
                        if (fresh || again) break;
                        reduce();
                        const bool up0 = top[0] > m[0] + kSlack, up1 = top[1] > m[1] + kSlack;
                        again = __any_sync(kFull, up0 || up1);
                        if (again) {  // 2^(-inf) = 0 where there was no maximum yet
                            alpha[0] = up0 ? ex2(m[0] - top[0]) : 1.0f;
                            alpha[1] = up1 ? ex2(m[1] - top[1]) : 1.0f;
                            if (up0) m[0] = top[0];
                            if (up1) m[1] = top[1];
                        }
                    } while (again);
                    l[0] = fmaf(l[0], alpha[0], add[0]);
                    l[1] = fmaf(l[1], alpha[1], add[1]);
                    if (again) {
                        // the last turn's product has run
                        if (!(ok = wait_all(&bar[L::PV_DONE + 2 * x + ((turns - 1) & 1)], ((turns - 1) >> 1) & 1))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[16];
                            tmem_ld_rows32(ts + kColO + x * D + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[(i >> 1) & 1]);
                            tmem_st_rows32(ts + kColO + x * D + c, o);
                        }
                    }
                    // the weights over the scores, which are read
                    tmem_st_pairs32(place, pk);
                    tmem_wait_st();
                }
                // stream 1: its O of the last unit of one tile is read
                if (x == 1 && t == 0 && joins > 0 && !(ok = wait_all(&bar[L::TAKEN + w8], (joins - 1) & 1))) break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[L::P_FULL + 2 * x + (turns & 1)]);
            }
            if (!ok) break;
            // ---- the end of the piece ----
            const bool any = s1 < n;  // this stream had steps
            if (any && !(ok = wait_all(&bar[L::PV_DONE + 2 * x + ((turns - 1) & 1)], ((turns - 1) >> 1) & 1))) break;
            tc_fence_after();
            float sum[2], fa[2], fb[2];  // O = fa O_x + fb O_1
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sum[i] = l[i];
                sum[i] += __shfl_xor_sync(kFull, sum[i], 1);
                sum[i] += __shfl_xor_sync(kFull, sum[i], 2);
                fa[i] = 1.0f;
                fb[i] = 0.0f;
            }
            if (!two) {
                if (x == 1) {
                    if (c4 == 0) {
                        stat[row0 + g8] = make_float2(m[0], sum[0]);
                        stat[row0 + g8 + 8] = make_float2(m[1], sum[1]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[L::STAT + w8]);
                    ++joins;
                    done_with(i);
                    continue;
                }
                if (!(ok = wait_all(&bar[L::STAT + w8], joins & 1))) break;
                ++joins;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 y = stat[row0 + g8 + 8 * i];
                    const float top = fmaxf(m[i], y.x);
                    fa[i] = m[i] == -INFINITY ? 0.0f : ex2(m[i] - top);
                    fb[i] = y.x == -INFINITY ? 0.0f : ex2(y.x - top);
                    sum[i] = sum[i] * fa[i] + y.y * fb[i];
                    m[i] = top;
                }
            }
            if (live) {
                const bool join = !two && n > 1, whole = p.whole();
                const int from = two ? x : n > 1 ? 0 : 1;  // a piece of one step is stream 1's alone
                const int slot = 2 * (int)blockIdx.x + (p.s0 == 0 ? 1 : 0);
                bool in[2];
                int64_t to[2];  // the row's place: in out, or in the slot
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float norm = whole ? (sum[i] > 0.0f ? vs / sum[i] : sum[i] == 0.0f ? 0.0f : sum[i]) : vs;
                    fa[i] = (from == x ? fa[i] : fb[i]) * norm;
                    fb[i] *= norm;
                    const int r = t0 + g8 + 8 * i;
                    in[i] = r < p.R;
                    to[i] = whole ? (((int64_t)p.row0 + node(i)) * a.n_q + p.g * G + min(r, p.R - 1) % G) * D
                                  : ((int64_t)slot * a.slot_rows + (r - p.r0)) * D;
                    if (!whole && in[i] && c4 == 0) a.ws_ml[(int64_t)slot * a.slot_rows + (r - p.r0)] = make_float2(m[i], sum[i]);
                }
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[16], o1[16];
                    tmem_ld_rows32(ts + kColO + from * D + c, o);
                    if (join) tmem_ld_rows32(ts + kColO + D + c, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {  // row i's columns c + 8 (j / 2) + 2 c4, + 1
                        const int i = j & 1;
                        float u = __uint_as_float(o[2 * j]) * fa[i], v = __uint_as_float(o[2 * j + 1]) * fa[i];
                        if (join) {
                            u = fmaf(fb[i], __uint_as_float(o1[2 * j]), u);
                            v = fmaf(fb[i], __uint_as_float(o1[2 * j + 1]), v);
                        }
                        if (!in[i]) continue;
                        const int64_t at = to[i] + c + 8 * (j >> 1) + 2 * c4;
                        if (whole) *reinterpret_cast<uint32_t *>(a.out + at) = pack_bf16x2(u, v);
                        else *reinterpret_cast<float2 *>(a.ws_o + at) = make_float2(u, v);
                    }
                }
            }
            if (!two) {  // stream 1 may go on
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[L::TAKEN + w8]);
            }
            done_with(i);
        }
        if (!ok) set_abort();
        else if (*odd_flag) {
            __syncwarp();
            add_odd_rows<D, G, F8>(a, *reinterpret_cast<const Slice *>(sm + L::kSlice), x, row0, lane);
        }
    }

    tc_fence_before();
    __syncthreads();  // every role is done with the tensor memory
    tc_fence_after();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ------------------------------------------------------------- the parts of cut units

struct MergeArgs {
    const Part *parts;
    const float2 *ws_ml;
    const float *ws_o;
    int slot_rows, n_q;
    __nv_bfloat16 *out;
};

constexpr int kMergeWarps = 8, kMergeBlocks = 4;  // of a slice

// Rows [i0, i0 + N) of a unit, those below i1: 32 parts at a time, a lane holding one's (m, l) of each row, and of the O
// 8 / N parts of all rows read at once.
template <int D, int G, int N>
__device__ __forceinline__ void join_rows(const MergeArgs &a, const Part &p, int first, int i0, int i1, int lane)
{
    constexpr int PL = D / 32;  // channels of a lane
    constexpr int U = 8 / N;
    auto at = [&](int w, int k) -> int64_t { return (int64_t)(k == 0 ? 2 * first + 1 : 2 * (first + k)) * a.slot_rows + i0 + w; };
    float o[N][PL] = {}, l[N] = {}, M[N];
#pragma unroll
    for (int w = 0; w < N; ++w) M[w] = -INFINITY;
    for (int k0 = 0; k0 <= p.more; k0 += 32) {
        const int n = min(32, p.more + 1 - k0);
        float2 y[N];
#pragma unroll
        for (int w = 0; w < N; ++w) y[w] = lane < n && i0 + w < i1 ? a.ws_ml[at(w, k0 + lane)] : make_float2(-INFINITY, 0.0f);
        float z[N][U][PL];
        auto load = [&](int k1) {
#pragma unroll
            for (int w = 0; w < N; ++w) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (k1 + u >= n || i0 + w >= i1) continue;
                    const float *src = a.ws_o + at(w, k0 + k1 + u) * D + lane * PL;
                    if constexpr (PL == 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(src);
                        z[w][u][0] = v.x; z[w][u][1] = v.y; z[w][u][2] = v.z; z[w][u][3] = v.w;
                    } else {
                        const float2 v = *reinterpret_cast<const float2 *>(src);
                        z[w][u][0] = v.x; z[w][u][1] = v.y;
                    }
                }
            }
        };
        load(0);  // (does not wait for the statistics)
        float f[N];
#pragma unroll
        for (int w = 0; w < N; ++w) {
            float top = y[w].x;
#pragma unroll
            for (int s = 16; s >= 1; s >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, s));
            const float was = M[w];
            M[w] = fmaxf(was, top);
            const float old = was == -INFINITY ? 0.0f : exp2f(was - M[w]);
            f[w] = y[w].x == -INFINITY ? 0.0f : exp2f(y[w].x - M[w]);
            float sum = y[w].y * f[w];
#pragma unroll
            for (int s = 16; s >= 1; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
            l[w] = l[w] * old + sum;
#pragma unroll
            for (int d = 0; d < PL; ++d) o[w][d] *= old;
        }
        for (int k1 = 0; k1 < n; k1 += U) {
            if (k1) load(k1);
#pragma unroll
            for (int w = 0; w < N; ++w) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float x = __shfl_sync(kFull, f[w], (k1 + u) & 31);
                    if (k1 + u >= n || i0 + w >= i1) continue;
#pragma unroll
                    for (int d = 0; d < PL; ++d) o[w][d] = fmaf(z[w][u][d], x, o[w][d]);
                }
            }
        }
    }
#pragma unroll
    for (int w = 0; w < N; ++w) {
        if (i0 + w >= i1) continue;
        const float inv = l[w] > 0.0f ? 1.0f / l[w] : l[w] == 0.0f ? 0.0f : l[w];
        const int r = p.r0 + i0 + w;
        __nv_bfloat16 *dst = a.out + (((int64_t)p.row0 + r / G) * a.n_q + p.g * G + r % G) * D + lane * PL;
        if constexpr (PL == 4)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(o[w][0] * inv, o[w][1] * inv), pack_bf16x2(o[w][2] * inv, o[w][3] * inv));
        else
            *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(o[w][0] * inv, o[w][1] * inv);
    }
}

// Blocks (c, ..) take a share of the rows of the unit that slice c has a part of and leaves to the next one: where it is
// cut once, all rows, up to four a warp at a time; where it is long, as many blocks as it has parts take few rows each.
// (Four blocks a slice, eight, two: one sequence of 32768 tokens 35.5, 36.1, 35.6 us a call, 64 trees on an E4M3 cache
// 132.3, 134.4, 134.3.  The first with 32 blocks for the rows of the unit that begins in a slice: 36.7.)
template <int D, int G>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const __grid_constant__ MergeArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const Part p = a.parts[blockIdx.x];
    if (p.more <= 0) return;
    const int rows = min(kUnitRows, p.R - p.r0);
    const int lo = rows * p.back / p.more, hi = rows * (p.back + 1) / p.more;
    const int warps = gridDim.y * kMergeWarps, at = blockIdx.y * kMergeWarps + (threadIdx.x >> 5), first = blockIdx.x - p.back;
    if (hi - lo <= warps) {
        if (lo + at < hi) join_rows<D, G, 1>(a, p, first, lo + at, hi, lane);
    } else if (hi - lo <= 2 * warps) {
        if (lo + 2 * at < hi) join_rows<D, G, 2>(a, p, first, lo + 2 * at, hi, lane);
    } else {
        for (int i = lo + 4 * at; i < hi; i += 4 * warps) join_rows<D, G, 4>(a, p, first, i, hi, lane);
    }
}

// ------------------------------------------------------------- launch

// The workspace of a call: parts, (m, l) and O of every slot.
struct Space {
    int slot_rows;
    size_t ml, o, bytes;
};
Space space_of(const pkv_pool *pool, int64_t n_rows, int G, int ctas)
{
    Space s;
    s.slot_rows = (int)std::min<int64_t>(kUnitRows, n_rows * G);
    const size_t slots = 2 * (size_t)ctas;
    s.ml = (ctas * sizeof(Part) + 255) / 256 * 256;
    s.o = s.ml + (slots * s.slot_rows * sizeof(float2) + 255) / 256 * 256;
    s.bytes = s.o + slots * s.slot_rows * (size_t)pool->d_head * sizeof(float);
    return s;
}

// The kernel's attributes are set, once per device.
template <int D, int G, bool F8>
pkv_status prepare(const pkv_pool *pool)
{
    static std::mutex mu;
    static bool ready[64];
    std::lock_guard<std::mutex> lock(mu);
    if (pool->device < 64 && ready[pool->device]) return PKV_OK;
    auto kern = tree_kernel<D, G, F8>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::bytes);
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return cuda_fail(e, "paged_tree_attention: kernel attributes");
    // (with fewer registers at the launch, the softmax warps would wait for theirs)
    if (fa.numRegs < Warps<F8>::kLaunchRegs)
        return fail(PKV_EUNSUPPORTED, "paged_tree_attention: built with %d registers a thread", fa.numRegs);
    if (pool->device < 64) ready[pool->device] = true;
    return PKV_OK;
}

template <int D, int G, bool F8>
pkv_status launch(pkv_pool *pool, const void *q, Args a, int ctas, cudaStream_t s)
{
    pkv_status st = prepare<D, G, F8>(pool);
    if (st != PKV_OK) return st;
    CUtensorMap tm_q;
    st = make_q_map(&tm_q, q, a.n_rows, a.n_q, D, G, kRows / G);
    if (st != PKV_OK) return st;
    {
        LaunchScope ls(pool, kDecode, s);
        cudaError_t e = launch_pdl(tree_kernel<D, G, F8>, dim3(ctas), dim3(Warps<F8>::kThreads), Layout<D>::bytes, s, tm_q,
                                   pool->tm_block, a);
        ls.done();
        if (e != cudaSuccess) return cuda_fail(e, "paged_tree_attention launch");
    }
    if (a.whole) return PKV_OK;
    MergeArgs m;
    m.parts = a.parts;
    m.ws_ml = a.ws_ml;
    m.ws_o = a.ws_o;
    m.slot_rows = a.slot_rows;
    m.n_q = a.n_q;
    m.out = a.out;
    LaunchScope ls(pool, kMerge, s);
    cudaError_t e = launch_pdl(tree_merge_kernel<D, G>, dim3(ctas, std::min(kMergeBlocks, (a.slot_rows + kMergeWarps - 1) / kMergeWarps)),
                               dim3(kMergeWarps * 32), 0, s, m);
    ls.done();
    if (e != cudaSuccess) return cuda_fail(e, "paged_tree_attention merge launch");
    return PKV_OK;
}

template <int D, bool F8>
pkv_status dispatch_g(pkv_pool *pool, const void *q, int G, const Args &a, int ctas, cudaStream_t s)
{
    switch (G) {
    case 1: return launch<D, 1, F8>(pool, q, a, ctas, s);
    case 2: return launch<D, 2, F8>(pool, q, a, ctas, s);
    case 4: return launch<D, 4, F8>(pool, q, a, ctas, s);
    case 8: return launch<D, 8, F8>(pool, q, a, ctas, s);
    }
    return fail(PKV_EUNSUPPORTED, "paged_tree_attention: group size %d unsupported (1, 2, 4 or 8)", G);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status paged_tree_reserve_workspace(pkv_pool *pool, int64_t n_rows, int32_t n_q)
{
    const char *who = "paged_tree_reserve_workspace";
    pkv_status st = check_step_args(pool, who, n_q, 1, 0, 1.0f);
    if (st != PKV_OK) return st;
    if (pool->dtype == PKV_INT4) return fail(PKV_EUNSUPPORTED, "%s: bf16 and FP8 pools only (not 4-bit)", who);
    if (n_rows < 0) return fail(PKV_EINVAL, "%s: n_rows < 0", who);
    st = check_pool_device(pool, who);
    if (st != PKV_OK) return st;
    return ensure_workspace(pool, space_of(pool, std::min<int64_t>(n_rows, kUnitRows), n_q / pool->n_kv, pool->num_sms).bytes);
}

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
    if (mask_words > kMaxWords) return fail(PKV_EUNSUPPORTED, "%s: mask_words %d > %d", who, mask_words, kMaxWords);
    if (batch == 0 || n_rows == 0) return PKV_OK;
    const int G = n_q / pool->n_kv;
    if (n_rows > INT32_MAX / G) return fail(PKV_EUNSUPPORTED, "%s: more than 2^31 query rows x group size", who);
    if (!q || !qo_indptr || !tree_mask || !block_tables || !context_lens || !out)
        return fail(PKV_EINVAL, "%s: NULL device pointer", who);
    if (((uintptr_t)q & 15u) || ((uintptr_t)out & 31u))
        return fail(PKV_EINVAL, "%s: q must be 16-byte and out 32-byte aligned", who);
    if (((uintptr_t)qo_indptr | (uintptr_t)block_tables | (uintptr_t)context_lens) & 3u || ((uintptr_t)tree_mask & 7u))
        return fail(PKV_EINVAL, "%s: indptr, tables and lengths must be 4-byte, masks 8-byte aligned", who);
    // a CTA stores a unit's rows while others have yet to read theirs: only a unit's own queries may be written over
    const size_t nout = (size_t)n_rows * n_q * pool->d_head * 2, nseq = (size_t)batch * 4;
    if (out != q && overlap(out, nout, q, nout)) return fail(PKV_EINVAL, "%s: out overlaps q without being q itself", who);
    if (overlap(out, nout, qo_indptr, nseq + 4) || overlap(out, nout, tree_mask, (size_t)n_rows * mask_words * 8) ||
        overlap(out, nout, block_tables, nseq * max_blocks_per_seq) || overlap(out, nout, context_lens, nseq) ||
        overlap(out, nout, pool->k, pool->alloc_bytes))
        return fail(PKV_EINVAL, "%s: out overlaps an input", who);
    st = check_pool_device(pool, who);
    if (st != PKV_OK) return st;
    // the most units and steps that the call can have: sequences may share rows (their indptr is not checked here)
    const int64_t most = std::min<int64_t>((int64_t)64 * mask_words, n_rows) * G;  // rows of a sequence and KV head
    const int64_t units = (int64_t)batch * pool->n_kv * ((most + kUnitRows - 1) / kUnitRows);
    const int64_t steps = (max_blocks_per_seq + kStepBlocks - 1) / kStepBlocks;
    if (units > INT32_MAX / (kCostTwo * steps + kCostUnit)) return fail(PKV_EUNSUPPORTED, "%s: too many rows x table entries", who);
    const int ctas = (int)std::min<int64_t>(pool->num_sms, units * steps);
    const Space sp = space_of(pool, n_rows, G, ctas);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = ensure_workspace(pool, sp.bytes, s, who);
    if (st != PKV_OK) return st;
    Args a;
    a.qo_indptr = qo_indptr;
    a.mask = reinterpret_cast<const uint32_t *>(tree_mask);
    a.words = mask_words;
    a.block_tables = block_tables;
    a.W = max_blocks_per_seq;
    a.context_lens = context_lens;
    a.batch = batch;
    a.n_q = n_q;
    a.n_kv = pool->n_kv;
    a.pool = static_cast<const uint8_t *>(pool->k);
    a.num_blocks = pool->num_blocks;
    a.n_rows = n_rows;
    a.oob_row = (int)(pool->num_blocks * pool->n_kv * 2 * kBlockSize);
    // (0 as 1e-30: the same scores to fp32, but -inf for hidden ones stays -inf)
    a.qscale = scale == 0.0f ? 1e-30f : scale * kLog2e;
    a.scales = pool->scales;
    a.whole = steps <= kWholeSteps;
    a.slot_rows = sp.slot_rows;
    uint8_t *ws = static_cast<uint8_t *>(pool->ws);
    a.parts = reinterpret_cast<Part *>(ws);
    a.ws_ml = reinterpret_cast<float2 *>(ws + sp.ml);
    a.ws_o = reinterpret_cast<float *>(ws + sp.o);
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.err = pool->err;
    const bool f8 = pool->dtype == PKV_FP8_E4M3;
    if (pool->d_head == 128)
        return f8 ? dispatch_g<128, true>(pool, q, G, a, ctas, s) : dispatch_g<128, false>(pool, q, G, a, ctas, s);
    return f8 ? dispatch_g<64, true>(pool, q, G, a, ctas, s) : dispatch_g<64, false>(pool, q, G, a, ctas, s);
}
