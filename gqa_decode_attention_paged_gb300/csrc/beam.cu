// Beam search's selection over beams and vocabulary.
//
// Mathematics.  Candidate (beam j, token t) of a search is worth
//   v = score_j + x_jt - lse_j,   lse_j = log sum_t exp x_jt;
// the k greatest are selected, equal ones by the lower j * vocab + t.  Within
// a row v grows with x, so a row's candidates are its k greatest logits, and
// only those need v.
//
// What bounds it: HBM, the logits read once, and the instructions: 11 per logit in
// bf16 (64 x 4 x 128256), 19 in fp32 where rows begin anywhere (32 x 10 x 100277),
// all steps counted, 43 and 47 % of the issue slots while an SM has work, which it
// has for 70 and 65 % of the time: with more rows than SMs they are not cut, and
// some SMs have one more than others.  One launch: a scan of the rows, cut into
// pieces so that every SM has three blocks where the rows are few, leaves each
// piece's maximum, sum of exponentials and k greatest logits; the block that is
// the last of a search to get there merges them (as a second launch that took the
// GPU as long, and the host 20 us a call instead of 15).
//
// Reading.  A piece streams through a ring of three parts of 16 KiB in shared
// memory (bulk copies: a vector a thread ahead kept 64 KiB in flight on an SM and
// waited for memory).  A row may begin anywhere.  Which thread adds which logits
// must depend neither on that nor on the row's number, or two beams with equal
// logits would get sums that differ in the last place, and equal continuations
// would not go to the lower beam.  So a thread takes the N elements from a
// multiple of N of the row on, out of two aligned vectors, and all rows are cut
// at the same places.
//
// Selecting while scanning.  From a piece's first part the threads' greatest
// logits, reduced to 4 k groups or more, give a bar: the k-th greatest group
// maximum, which at least k logits reach.  The warps then go through the rest
// each for itself, and note the vectors that have a logit above the bar: about
// 1.15 k (n / n_1 - 1) where the logits come in any order (n_1: those that the
// bar is from).  Before that comes near what can be noted, the noted logits are
// taken, and give the next bar (16 searches x 16 beams x 128256 in fp32, k = 24,
// 32, 64: 129, 134, 68..185 us without, 49, 49, 69 so).  At the end the logits of
// the noted vectors are taken out of them.  Where they rise along the row, or
// many equal the bar, the notes or what is in them can be too many; the piece is
// then read again, and every part raises the bar first: what reaches it belongs
// to k groups, so it fits whatever the data.  Keys (logit as an ordered integer,
// then the lower index) are unique, so ties need no care and results do not
// depend on the order of arrival.
//
// Accuracy.  Candidates of different beams may lie arbitrarily close, so what
// decides between them is held in more than 32 bits: the exponentials are
// 32-bit (of x - m, exact near the maximum, where they count), a thread adds 16
// or 32 of them in 32 bits and those sums with what their additions lose, all
// further sums are 64-bit integers (2^-40 of the largest term), and
// the logarithm and v are doubles.
#include <algorithm>
#include <climits>
#include <math.h>
#include <mutex>

#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;                         // 16-byte vectors of a thread and part
constexpr int kPartVecs = kVecs * kThreads;
constexpr int kStages = 3;
constexpr int kBlocksPerSm = 3;
constexpr int kStageBytes = kPartVecs * 16 + 128; // with the vector behind it
constexpr int kMaxK = 64, kMaxBeams = 64;
constexpr int kPartKeys = 2048;                  // of a part, that reach its bar, at most
constexpr int kCap = 2304;                       // keys the buffer holds: those, k kept ones, some more
constexpr int kNotes = 1280;                     // vectors that can be noted
// The bar is raised after 1 + kRaise / k parts, then whenever there were as many times the parts before: about 1.15 kRaise
// are noted until then, give or take 1 / sqrt(k) of it, as the bar is the k-th of a sample.
constexpr int kRaise = 512;

// How rows are cut: piece i of a row has parts [first(i), first(i + 1)).
struct Cut {
    int parts, pieces;
    __host__ __device__ int first(int i) const { return (int)((int64_t)parts * i / pieces); }
};

struct Args {
    const void *logits;
    int64_t stride;       // elements between rows
    int vocab, k;
    Cut cut;
    const float *scores;  // [batch][beams]
    uint64_t *keys;       // [rows][cut.pieces][k], greatest first, 0: none
    float *top;           // [rows][cut.pieces] maximum
    double *sum;          // [rows][cut.pieces] sum of exp(x - maximum); NaN where the piece holds a NaN or +infinity
    unsigned *tickets;    // [batch] blocks of a search that have left their lists; 0 before and after a call
    int32_t *tokens, *parents;  // [batch][k]
    float *out;                 // [batch][k]
    unsigned *err;
};

// The order of keys is that of the logits, then of the lower index; 0 is below all of them.
__device__ __forceinline__ uint64_t key_of(float x, int index)
{
    const uint32_t u = __float_as_uint(x + 0.0f);  // (-0 counts as +0)
    const uint32_t o = u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
    return ((uint64_t)o << 32) | (0xffffffffu - (uint32_t)index);
}
__device__ __forceinline__ float logit_of(uint64_t key)
{
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ int index_of(uint64_t key) { return (int)(0xffffffffu - (uint32_t)key); }

template <typename T>
struct Elems;
template <>
struct Elems<__nv_bfloat16> {
    static constexpr int N = 8;  // of a vector
    static constexpr uint32_t kLow = 0xff80ff80u;  // -infinity
    static __device__ __forceinline__ void widen(const uint4 &v, float (&x)[8])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_f32x2(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <>
struct Elems<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kLow = 0xff800000u;
    static __device__ __forceinline__ void widen(const uint4 &v, float (&x)[4])
    {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
};

struct Shared {
    alignas(128) uint8_t ring[kStages][kStageBytes];
    uint64_t full[kStages];
    int readers[kStages];  // warps that have read a stage's part
    uint64_t buf[kCap];
    uint64_t group[kThreads];
    int note[kNotes];
    int notes;         // (those past kNotes are not there)
    uint64_t bar;      // keys below it are not among the k greatest
    uint64_t sums[kWarps];
    float tops[kWarps];
    int n;             // keys in buf (those past kCap are not there)
    bool last;         // the block merges
};

__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// Raises sh.bar to the k-th greatest of the groups' greatest keys (of `mine`, 0: none; 8 p groups of 32 / p
// neighbouring threads), if that many groups have one.  At least k of the threads' keys reach it, and those that
// do belong to k groups.
__device__ __forceinline__ void raise_bar(Shared &sh, uint64_t mine, int k, int p)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int size = 32 / p;
    for (int o = size / 2; o >= 1; o >>= 1) mine = max64(mine, __shfl_xor_sync(kFull, mine, o));
    if (lane % size == 0) sh.group[warp * p + lane / size] = mine;
    __syncthreads();
    const int groups = kWarps * p;
    if (tid < groups) {
        const uint64_t x = sh.group[tid];
        int rank = 0;
        for (int i = 0; i < groups; ++i) rank += sh.group[i] > x;
        if (x && rank == k - 1 && x > sh.bar) sh.bar = x;  // (one thread: keys are unique)
    }
    __syncthreads();
}

// Keeps the keys of buf (n, known to all threads) that can be among the k greatest, until `most` at most are
// left; how many are.
__device__ __forceinline__ int thin_out(Shared &sh, int n, int k, int p, int most)
{
    constexpr int U = kCap / kThreads;
    const int tid = threadIdx.x;
    while (n > most) {
        uint64_t x[U], mine = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = u * kThreads + tid;
            x[u] = i < n ? sh.buf[i] : 0;
            mine = max64(mine, x[u]);
        }
        raise_bar(sh, mine, k, p);  // (its barriers: every thread has its keys)
        if (tid == 0) sh.n = 0;
        __syncthreads();
        const uint64_t bar = sh.bar;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (x[u] && x[u] >= bar) sh.buf[atomicAdd(&sh.n, 1)] = x[u];
        __syncthreads();
        n = sh.n;
        __syncthreads();  // (read by all before anyone adds to it)
    }
    return n;
}

// A continuation: its worth as an ordered integer (0: none), then what settles equal worths: the lower beam, then the
// greater logit (a beam's different logits may have one worth in 64 bits), then the lower token.
struct Cand {
    uint64_t value, tie;
    __device__ __forceinline__ bool above(const Cand &y) const { return value != y.value ? value > y.value : tie > y.tie; }
};
constexpr int kTokenBits = 22;
__device__ __forceinline__ Cand shfl_xor(const Cand &x, int o)
{
    return {__shfl_xor_sync(kFull, x.value, o), __shfl_xor_sync(kFull, x.tie, o)};
}

constexpr int kHold = 8;                         // continuations of a thread, at a time
constexpr int kMergeKeep = 1024;                 // kept between rounds
constexpr int kMergeCap = kMergeKeep + kHold * kThreads / 4;
constexpr int kFewLists = 8;                     // bisected by every continuation: 4 lists of 8 take 11.6 us a call, with a bar 12.7; 16: 13.7, 11.5

struct MergeShared {
    Cand buf[kMergeCap];
    Cand group[kThreads];
    Cand bar;
    int n;
    double shift[kMaxBeams];   // score - log of the sum of exp(x - m); NaN: no continuations
    float highest[kMaxBeams];  // m: v = (x - m) + shift, in which large logits cost nothing
};

// The k-th greatest of the groups' greatest continuations, if as many groups have one: as raise_bar, 8 p groups.
__device__ __forceinline__ void raise_bar(MergeShared &sh, Cand mine, int k, int p)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, size = 32 / p;
    for (int o = size / 2; o >= 1; o >>= 1) {
        const Cand y = shfl_xor(mine, o);
        if (y.above(mine)) mine = y;
    }
    if (lane % size == 0) sh.group[warp * p + lane / size] = mine;
    __syncthreads();
    const int groups = kWarps * p;
    if (tid < groups) {
        const Cand x = sh.group[tid];
        int rank = 0;
        for (int i = 0; i < groups; ++i) rank += sh.group[i].above(x);
        if (x.value && rank == k - 1 && x.above(sh.bar)) sh.bar = x;  // (one thread: continuations are unique)
    }
    __syncthreads();
}

// One search: its beams' log-sums, the worth of its lists' continuations, and the k greatest of them, found as the
// scan finds a row's (k rounds over the lists' heads took 0.65 us each).
__device__ __noinline__ void merge(MergeShared &sh, const Args &a, int beams, int64_t item)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pieces = a.cut.pieces, per_beam = pieces * a.k, total = beams * per_beam;
    const uint64_t *keys = a.keys + item * total;
    if (tid == 0) {
        sh.bar = {0, 0};
        sh.n = 0;
    }
    auto key_at = [&](int i) -> uint64_t { return i < total ? __ldcg(keys + i) : 0; };  // (from the L2: other blocks wrote them)
    uint64_t held = key_at(tid);  // (read while the log-sums are formed)
    // a lane a piece, as many beams a warp as its lanes have room for
    int group = 1;
    while (group < pieces && group < 32) group *= 2;
    for (int j0 = warp * (32 / group); j0 < beams; j0 += kWarps * (32 / group)) {
        const int j = j0 + lane / group, first = lane % group;
        const bool there = j < beams;
        const int64_t row = item * beams + j, l0 = row * pieces;
        const float sc = there ? a.scores[row] : -INFINITY;
        const float t0 = there && first < pieces ? __ldcg(a.top + l0 + first) : -INFINITY;
        const double x0 = there && first < pieces ? __ldcg(a.sum + l0 + first) : 0.0;
        float M = t0;
        for (int i = first + 32; there && i < pieces; i += 32) M = fmaxf(M, __ldcg(a.top + l0 + i));
        for (int o = group / 2; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
        // (of an infinite maximum the sum is NaN)
        auto scaled = [&](float t, double x) { return t == M || x != x ? x : t == -INFINITY ? 0.0 : x * exp((double)t - (double)M); };
        double s = scaled(t0, x0);
        for (int i = first + 32; there && i < pieces; i += 32) s += scaled(__ldcg(a.top + l0 + i), __ldcg(a.sum + l0 + i));
        for (int o = group / 2; o >= 1; o >>= 1) s += __shfl_xor_sync(kFull, s, o);  // (lanes past the pieces hold 0)
        if (!there || first) continue;
        const bool odd = sc != -INFINITY && (s != s || sc != sc || sc == INFINITY);
        if (odd) atomicOr(a.err, PKV_DEVERR_NAN);
        sh.shift[j] = odd || sc == -INFINITY || M == -INFINITY ? (double)NAN : (double)sc - log(s);
        sh.highest[j] = M;
    }
    __syncthreads();
    auto worth = [&](uint64_t key, int i) -> Cand {
        if (!key) return {0, 0};
        const int j = i / per_beam;
        const double v = ((double)logit_of(key) - (double)sh.highest[j]) + sh.shift[j];
        if (v != v) return {0, 0};
        const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
        return {u ^ ((u >> 63) ? ~0ull : 1ull << 63),
                ((uint64_t)(kMaxBeams - 1 - j) << (32 + kTokenBits)) | ((key >> 32) << kTokenBits) |
                    (uint64_t)((1 << kTokenBits) - 1 - index_of(key))};
    };
    auto put = [&](int rank, const Cand &x) {
        const int64_t o = item * a.k + rank;
        const uint64_t u = x.value ^ ((x.value >> 63) ? 1ull << 63 : ~0ull);
        a.tokens[o] = (1 << kTokenBits) - 1 - (int)(x.tie & ((1 << kTokenBits) - 1));
        a.parents[o] = kMaxBeams - 1 - (int)(x.tie >> (32 + kTokenBits));
        a.out[o] = (float)__longlong_as_double((long long)u);
    };
    auto put_none = [&](int rank) {  // no continuation is left for this place
        const int64_t o = item * a.k + rank;
        a.tokens[o] = a.parents[o] = -1;
        a.out[o] = -INFINITY;
    };
    const int lists = beams * pieces;
    if (lists <= kFewLists && total <= kThreads) {
        // a thread a continuation: its rank is its place in its list and, by bisection, in every other one
        const Cand x = worth(held, tid);
        sh.buf[tid] = x;
        const int live = __syncthreads_count(x.value != 0);
        if (tid >= live && tid < a.k) put_none(tid);
        if (!x.value) return;
        const int own = tid / a.k;
        int rank = tid - own * a.k;
        // (not unrolled: code that runs once waits for its instructions)
#pragma unroll 1
        for (int l = 0; l < lists; ++l) {
            if (l == own) continue;
            int lo = 0, hi = a.k;  // elements [0, lo) are above x, [hi, k) are not
#pragma unroll 1
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (sh.buf[l * a.k + mid].above(x)) lo = mid + 1;
                else hi = mid;
            }
            rank += lo;
        }
        if (rank < a.k) put(rank, x);
        return;
    }
    // kHold keys a thread at a time: at least k of them reach the bar, and those that do are of k groups
    const int p = a.k <= 4 ? 2 : a.k <= 8 ? 4 : a.k <= 16 ? 8 : a.k <= 32 ? 16 : 32;  // groups of a warp
    auto greatest = [&](const Cand (&c)[kHold]) -> Cand {
        Cand top = c[0];
#pragma unroll
        for (int i = 1; i < kHold; ++i)
            if (c[i].above(top)) top = c[i];
        return top;
    };
    // keeps those of c that reach the bar: of k groups of 32 / p threads with kHold each, 512 at most
    auto keep = [&](const Cand (&c)[kHold]) {
        const Cand bar = sh.bar;
#pragma unroll
        for (int i = 0; i < kHold; ++i)
            if (c[i].value && !bar.above(c[i])) sh.buf[atomicAdd(&sh.n, 1)] = c[i];
        __syncthreads();
    };
    for (int base = 0; base < total; base += kHold * kThreads) {
        Cand c[kHold];
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int at = base + i * kThreads + tid;
            c[i] = worth(base == 0 && i == 0 ? held : key_at(at), at);
        }
        raise_bar(sh, greatest(c), a.k, p);
        keep(c);
        // fewer again, before the next ones or the end
        for (int n = sh.n; n > (base + kHold * kThreads < total ? kMergeKeep : kThreads);) {
            __syncthreads();  // (n is read)
#pragma unroll
            for (int i = 0; i < kHold; ++i) c[i] = i * kThreads + tid < n ? sh.buf[i * kThreads + tid] : Cand{0, 0};
            raise_bar(sh, greatest(c), a.k, p);
            if (tid == 0) sh.n = 0;
            __syncthreads();
            keep(c);
            n = sh.n;
        }
        __syncthreads();
    }
    // ---- in order ----
    const int n = sh.n;
    if (tid < n) {
        const Cand x = sh.buf[tid];
        int rank = 0;
        for (int i = 0; i < n; ++i) rank += sh.buf[i].above(x);
        if (rank < a.k) put(rank, x);
    } else if (tid < a.k) {
        put_none(tid);
    }
}

// A row of logits as 16-byte aligned vectors u, elements u N - lead .. + N - 1.
template <typename T>
struct Row {
    using El = Elems<T>;
    static constexpr int N = El::N;
    const T *x;
    int vocab, lead;  // elements before the row in its first aligned vector

    // vectors [inner0(), inner1()) are inside the row
    __device__ __forceinline__ int inner0() const { return lead ? 1 : 0; }
    __device__ __forceinline__ int inner1() const { return (int)(((int64_t)vocab + lead) / N); }
    __device__ __forceinline__ bool inside(int u) const { return u >= inner0() && u < inner1(); }
    __device__ __forceinline__ const T *at(int u) const { return x + ((int64_t)u * N - lead); }
    // a vector that the row begins or ends in, or one behind it
    __device__ uint4 edge(int u) const
    {
        const int i = u * N - lead;
        uint32_t w[4] = {El::kLow, El::kLow, El::kLow, El::kLow};
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (i + e < 0 || i + e >= vocab) continue;
            if constexpr (N == 4) {
                w[e] = __float_as_uint(x[i + e]);
            } else {
                const uint32_t h = __bfloat16_as_ushort(x[i + e]);
                w[e / 2] = e % 2 ? (w[e / 2] & 0xffffu) | (h << 16) : (w[e / 2] & 0xffff0000u) | h;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // elements u N .. + N - 1, out of vectors u and u + 1
    __device__ __forceinline__ uint4 line_up(const uint4 &r, const uint4 &next) const
    {
        uint32_t w[8] = {r.x, r.y, r.z, r.w, next.x, next.y, next.z, next.w};
        const int words = lead * (int)sizeof(T) / 4;
        if (words & 2) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (words & 1) {
#pragma unroll
            for (int i = 0; i < 7; ++i) w[i] = w[i + 1];
        }
        if (N == 8 && (lead & 1)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    template <typename Get>
    __device__ __forceinline__ uint4 elements(int u, Get &&get) const
    {
        const uint4 r = inside(u) ? get(u) : edge(u);
        if (!lead) return r;
        return line_up(r, inside(u + 1) ? get(u + 1) : edge(u + 1));
    }
};

// The greatest of a vector's logits; a NaN is passed over.
template <typename T>
__device__ __forceinline__ float greatest_of(const uint4 &v)
{
    if constexpr (sizeof(T) == 2) {
        auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
        const __nv_bfloat162 m = __hmax2(__hmax2(h(v.x), h(v.y)), __hmax2(h(v.z), h(v.w)));
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
}

// A thread's greatest logit so far and the sum of exp(x - m), as s + lost: a row of 2^22 logits in one piece is 1024
// parts, which plain 32-bit additions would round as often.
struct Sum {
    float m = -INFINITY, s = 0.0f, lost = 0.0f;
    // a part's vectors, with the greatest logit top
    template <typename T>
    __device__ __forceinline__ void add(const uint4 (&v)[kVecs], float top)
    {
        constexpr int N = Elems<T>::N;
        if (top > m) {
            const float less = m == -INFINITY ? 1.0f : ex2((m - top) * kLog2e);
            s *= less;
            lost *= less;
            m = top;
        }
        // (of x - m, not of x log2(e) - m log2(e), whose second product's rounding would be in every term alike)
        const float neg = m == -INFINITY ? 0.0f : -m;
        float2 part = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float x[N];
            Elems<T>::widen(v[i], x);
#pragma unroll
            for (int e = 0; e < N; e += 2) {
                const float2 d = fmul2(fadd2(make_float2(x[e], x[e + 1]), make_float2(neg, neg)), make_float2(kLog2e, kLog2e));
                part = fadd2(part, make_float2(ex2(d.x), ex2(d.y)));
            }
        }
        // (the greater of the two is not known: the two-sided form of the error of an addition)
        const float add = part.x + part.y, t = __fadd_rn(s, add), b = __fsub_rn(t, s);
        lost = __fadd_rn(lost, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(add, b)));
        s = t;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) beam_select_kernel(const __grid_constant__ Args a)
{
    using El = Elems<T>;
    constexpr int N = El::N;
    extern __shared__ __align__(128) uint8_t beam_smem[];
    Shared &sh = *reinterpret_cast<Shared *>(beam_smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        sh.n = sh.notes = 0;
        sh.bar = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            sh.readers[i] = 0;
        }
        fence_mbarrier_init();
    }
    griddep_wait();
    griddep_launch_dependents();
    const int k = a.k;
    // groups of a warp: 4 k in all, and k of them have k (32 / p) threads' 32 logits, kPartKeys at most
    const int p = k <= 4 ? 2 : k <= 8 ? 4 : k <= 16 ? 8 : k <= 32 ? 16 : 32;
    const uint64_t policy = l2_policy_evict_first();
    const int piece = blockIdx.x, r0 = a.cut.first(piece), parts = a.cut.first(piece + 1) - r0;
    const int64_t row = (int64_t)blockIdx.y * gridDim.z + blockIdx.z;  // (search, beam)
    Row<T> rw;
    rw.x = static_cast<const T *>(a.logits) + row * a.stride;
    rw.vocab = a.vocab;
    rw.lead = (int)(((uintptr_t)rw.x & 15u) / sizeof(T));
    // part q into its stage: the vectors that are inside the row, and the one behind the part's last
    auto issue = [&](int q) {
        const int v0 = (r0 + q) * kPartVecs, st = q % kStages;
        const int u0 = max(v0, rw.inner0()), u1 = min(v0 + kPartVecs + (rw.lead ? 1 : 0), rw.inner1());
        const uint32_t bytes = u1 > u0 ? 16u * (uint32_t)(u1 - u0) : 0u;
        mbar_arrive_expect_tx(&sh.full[st], bytes);
        if (bytes) bulk_g2s(sh.ring[st] + (u0 - v0) * 16, rw.at(u0), bytes, &sh.full[st], policy);
    };
    if (tid == 0)
        for (int q = 0; q < min(parts, kStages); ++q) issue(q);
    __syncthreads();
    bool ok = true;
    // this thread's vectors of part q
    auto fetch = [&](int q, uint4 (&v)[kVecs]) {
        const int st = q % kStages, v0 = (r0 + q) * kPartVecs;
        ok = ok && __all_sync(kFull, mbar_wait_bounded(&sh.full[st], (q / kStages) & 1));
        const uint32_t ring = smem_u32(sh.ring[st]);
        const bool inner = v0 >= rw.inner0() && v0 + kPartVecs < rw.inner1();
        if (inner) {  // (and the vector behind the part is)
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i] = lds128(ring + (i * kThreads + tid) * 16);
            if (rw.lead) {
#pragma unroll
                for (int i = 0; i < kVecs; ++i) v[i] = rw.line_up(v[i], lds128(ring + (i * kThreads + tid + 1) * 16));
            }
        } else {
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                v[i] = rw.elements(v0 + i * kThreads + tid, [&](int u) { return lds128(ring + (u - v0) * 16); });
        }
        // the last warp to have read a part has its stage filled again: none waits for another
        __threadfence_block();
        __syncwarp();
        if (lane == 0 && atomicAdd(&sh.readers[st], 1) == kWarps - 1) {
            sh.readers[st] = 0;
            if (q + kStages < parts) {
                __threadfence_block();
                fence_proxy_async_smem();
                issue(q + kStages);
            }
        }
    };
    static_assert(kVecs == 4, "");
    auto greatest = [&](const uint4 (&v)[kVecs], float (&tops)[kVecs]) -> float {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) tops[i] = greatest_of<T>(v[i]);
        return fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    };
    // index in the row of the first element of this thread's vector i of part q
    auto first = [&](int q, int i) -> int { return ((r0 + q) * kPartVecs + i * kThreads + tid) * N; };
    // the key of a thread's greatest logit: of equal ones the first
    auto key_at = [&](const uint4 (&v)[kVecs], int q, float top) -> uint64_t {
        if (!(top > -INFINITY)) return 0;
        int at = 0;
#pragma unroll
        for (int i = kVecs - 1; i >= 0; --i) {
            float x[N];
            El::widen(v[i], x);
#pragma unroll
            for (int e = N - 1; e >= 0; --e) at = x[e] == top ? i * (kThreads * N) + e : at;
        }
        return key_of(top, first(q, 0) + at);
    };
    // adds a vector's logits that reach the bar to the buffer
    auto add_keys = [&](const uint4 &w, int at0, uint64_t bar) {
        float x[N];
        El::widen(w, x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (!(x[e] > -INFINITY)) continue;
            const uint64_t key = key_of(x[e], at0 + e);
            if (key < bar) continue;
            const int at = atomicAdd(&sh.n, 1);
            if (at < kCap) sh.buf[at] = key;
        }
    };
    auto note = [&](int q, int i) {
        const int at = atomicAdd(&sh.notes, 1);
        if (at < kNotes) sh.note[at] = first(q, i);
    };
    Sum sum;
    uint4 v[kVecs];
    float tops[kVecs];
    fetch(0, v);
    float top = greatest(v, tops);
    raise_bar(sh, key_at(v, 0, top), k, p);
    uint64_t bar = sh.bar;
    float high = bar ? logit_of(bar) : -INFINITY;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
        if (tops[i] > -INFINITY && tops[i] >= high) note(0, i);
    sum.add<T>(v, top);
    auto read = [&](int i0) -> uint4 { return rw.elements(i0 / N, [&](int u) { return ldg_nc_v4(rw.at(u)); }); };
    // ---- the rest of the piece, every warp for itself ----
    int raise = 1 + kRaise / k;
    for (int q = 1; q < parts; ++q) {
        if (q == raise) {  // the notes taken so far give a higher bar
            raise = q + q * (kRaise / k);
            __syncthreads();
            const int notes = sh.notes;
            if (notes <= kNotes) {
                for (int i = tid; i < notes; i += kThreads) add_keys(read(sh.note[i]), sh.note[i], bar);
                __syncthreads();
                const int have = sh.n;
                __syncthreads();
                if (have <= kCap) {  // (else the piece is read again, below)
                    thin_out(sh, have, k, p, kMaxK);
                    if (tid == 0) sh.notes = 0;
                    __syncthreads();
                    bar = sh.bar;
                    high = bar ? logit_of(bar) : -INFINITY;
                }
            }
        }
        fetch(q, v);
        top = greatest(v, tops);
        if (top > high) {  // (an equal one has a greater index than the bar's)
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                if (tops[i] > high) note(q, i);
        }
        sum.add<T>(v, top);
    }
    // ---- the piece's maximum and sum ----
    float M = sum.m;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    if (lane == 0) sh.tops[warp] = M;
    const bool bad = __syncthreads_or(!(sum.s < INFINITY));  // (the sum of a NaN or an infinite logit is NaN)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh.tops[w]);
    uint64_t f = 0;  // this thread's sum in units of 2^-40
    if (!bad && sum.m > -INFINITY) {
        const float unit = ex2((sum.m - M) * kLog2e) * 0x1p40f;
        f = (uint64_t)(__float2ll_rn(sum.s * unit) + __float2ll_rn(sum.lost * unit));
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) f += __shfl_xor_sync(kFull, f, o);
    if (lane == 0) sh.sums[warp] = f;
    const int notes = sh.notes;
    if (notes <= kNotes)
        for (int i = tid; i < notes; i += kThreads) add_keys(read(sh.note[i]), sh.note[i], bar);
    __syncthreads();
    int n = sh.n;
    __syncthreads();
    if (notes > kNotes || n > kCap) {  // too many: the piece again, part by part
        if (tid == 0) {
            sh.n = 0;
            sh.bar = 0;
        }
        __syncthreads();
        for (int q = 0; q < parts; ++q) {
            const int have = sh.n;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i] = read(first(q, i));
            raise_bar(sh, key_at(v, q, greatest(v, tops)), k, p);
            if (have + kPartKeys > kCap) thin_out(sh, have, k, p, kMaxK);
            const uint64_t now = sh.bar;
#pragma unroll 1
            for (int i = 0; i < kVecs; ++i) add_keys(i == 0 ? v[0] : i == 1 ? v[1] : i == 2 ? v[2] : v[3], first(q, i), now);
            __syncthreads();
        }
        n = sh.n;
        __syncthreads();
    }
    n = thin_out(sh, n, k, p, kThreads);
    const int64_t list = row * a.cut.pieces + piece;
    if (tid == 0) {
        for (int w = 1; w < kWarps; ++w) f += sh.sums[w];
        a.top[list] = M;
        a.sum[list] = bad ? (double)NAN : (double)f * 0x1p-40;
    }
    // ---- its k greatest, in order ----
    if (tid < n) {
        const uint64_t x = sh.buf[tid];
        int rank = 0;
        for (int i = 0; i < n; ++i) rank += sh.buf[i] > x;
        if (rank < k) a.keys[list * k + rank] = x;
    } else if (tid < k) {
        a.keys[list * k + tid] = 0;
    }
    // ---- the last block of the search takes all its lists ----
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        unsigned *ticket = a.tickets + blockIdx.y;
        const unsigned blocks = gridDim.x * gridDim.z;
        sh.last = atomicAdd(ticket, 1u) == blocks - 1;
        if (sh.last) *ticket = 0;  // (nobody else comes)
        __threadfence();
    }
    __syncthreads();
    if (!ok) {
        if (lane == 0) atomicOr(a.err, PKV_DEVERR_TIMEOUT);
        if (warp == 0)  // copies in flight land before the block exits
            for (int q = max(0, parts - kStages); q < parts; ++q) mbar_wait_bounded(&sh.full[q % kStages], (q / kStages) & 1);
    }
    if (sh.last) {
        __syncthreads();  // (read by all: the merge has the same memory)
        merge(*reinterpret_cast<MergeShared *>(beam_smem), a, (int)gridDim.z, blockIdx.y);
    }
}

static_assert(kBlocksPerSm * (sizeof(Shared) + 1024) <= 232448, "fewer blocks would fit on an SM");
static_assert(sizeof(MergeShared) <= sizeof(Shared), "");

// Pieces of a row: as many as all blocks that run at once have room for, of two parts each at least (the bar comes
// from the first).  Shorter rows are not cut: 4 and 8 beams x 32000 in bf16, four parts, take 11.6 and 14.3 us whole,
// 12.3 and 16.2 in two; sixteen parts (128256), where the rows are few, 12.7 and 16.2 in eight, 16.2 and 16.0 in four.
constexpr int kCutParts = 6;
Cut cut_of(const pkv_pool *pool, int64_t rows, int vocab, int elem)
{
    const int part = kPartVecs * (16 / elem);
    Cut c;
    c.parts = (vocab + part - 1) / part;
    const int64_t room = (int64_t)kBlocksPerSm * pool->num_sms / std::max<int64_t>(1, rows);
    c.pieces = c.parts < kCutParts ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(room, c.parts / 2));
    return c;
}

// The kernel's shared memory is allowed, once per device.
pkv_status prepare_scan(const pkv_pool *pool)
{
    static std::mutex mu;
    static bool ready[64];
    std::lock_guard<std::mutex> lock(mu);
    if (pool->device < 64 && ready[pool->device]) return PKV_OK;
    cudaError_t e = cudaFuncSetAttribute(beam_select_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(beam_select_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
    if (e != cudaSuccess) return cuda_fail(e, "paged_beam_select: kernel attributes");
    if (pool->device < 64) ready[pool->device] = true;
    return PKV_OK;
}

size_t beam_bytes(int64_t rows, const Cut &c, int k) { return (size_t)rows * c.pieces * (8 * (size_t)k + 16); }

pkv_status check_beam(const pkv_pool *pool, const char *who, int batch, int beams, int vocab, int k, int type)
{
    if (!pool) return fail(PKV_EINVAL, "%s: NULL pool", who);
    if (type != PKV_LOGITS_BF16 && type != PKV_LOGITS_F32) return fail(PKV_EINVAL, "%s: unknown logits type %d", who, type);
    if (batch < 0 || batch > kMaxBatch) return fail(PKV_EINVAL, "%s: batch %d out of range", who, batch);
    if (beams < 1 || beams > kMaxBeams) return fail(PKV_EUNSUPPORTED, "%s: %d beams (1 .. %d)", who, beams, kMaxBeams);
    if (k < 1 || k > kMaxK) return fail(PKV_EUNSUPPORTED, "%s: k = %d (1 .. %d)", who, k, kMaxK);
    if (vocab < 1) return fail(PKV_EINVAL, "%s: vocab %d", who, vocab);
    if (vocab > (1 << 22)) return fail(PKV_EUNSUPPORTED, "%s: vocab %d > 2^22", who, vocab);
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status paged_beam_reserve_workspace(pkv_pool *pool, int32_t batch, int32_t beams, int32_t vocab, int32_t k)
{
    const char *who = "paged_beam_reserve_workspace";
    pkv_status st = check_beam(pool, who, batch, beams, vocab, k, PKV_LOGITS_BF16);
    if (st == PKV_OK) st = check_pool_device(pool, who);
    if (st != PKV_OK) return st;
    size_t most = 0;
    for (int b = 1; b <= batch; ++b)  // (rows of smaller calls have more pieces)
        for (int elem : {2, 4}) {
            const int64_t rows = (int64_t)b * beams;
            most = std::max(most, beam_bytes(rows, cut_of(pool, rows, vocab, elem), k));
        }
    return ensure_workspace(pool, most);
}

extern "C" pkv_status paged_beam_select(pkv_pool *pool, const void *logits, int32_t type, int64_t row_stride,
                                        const float *scores, int32_t batch, int32_t beams, int32_t vocab, int32_t k,
                                        int32_t *tokens, int32_t *parents, float *out_scores, void *stream)
{
    const char *who = "paged_beam_select";
    pkv_status st = check_beam(pool, who, batch, beams, vocab, k, type);
    if (st != PKV_OK) return st;
    if (row_stride < vocab) return fail(PKV_EINVAL, "%s: row_stride %lld < vocab %d", who, (long long)row_stride, vocab);
    if (batch == 0) return PKV_OK;
    if (!logits || !scores || !tokens || !parents || !out_scores) return fail(PKV_EINVAL, "%s: NULL device pointer", who);
    const int elem = type == PKV_LOGITS_F32 ? 4 : 2;
    if (((uintptr_t)logits & (elem - 1)) ||
        (((uintptr_t)scores | (uintptr_t)tokens | (uintptr_t)parents | (uintptr_t)out_scores) & 3u))
        return fail(PKV_EINVAL, "%s: arrays must be aligned to their elements", who);
    const int64_t rows = (int64_t)batch * beams;
    if (row_stride > ((int64_t)1 << 40) / rows) return fail(PKV_EUNSUPPORTED, "%s: row_stride too large", who);
    const size_t nout = (size_t)batch * k * 4, nlog = ((size_t)(rows - 1) * row_stride + vocab) * elem;
    const void *outs[3] = {tokens, parents, out_scores};
    for (int i = 0; i < 3; ++i) {
        if (overlap(outs[i], nout, logits, nlog) || overlap(outs[i], nout, scores, (size_t)rows * 4))
            return fail(PKV_EINVAL, "%s: an output overlaps an input", who);
        if (overlap(outs[i], nout, outs[(i + 1) % 3], nout)) return fail(PKV_EINVAL, "%s: the outputs overlap", who);
    }
    st = check_pool_device(pool, who);
    if (st != PKV_OK) return st;
    const Cut cut = cut_of(pool, rows, vocab, elem);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = ensure_workspace(pool, beam_bytes(rows, cut, k), s, who);
    if (st != PKV_OK) return st;
    st = prepare_scan(pool);
    if (st != PKV_OK) return st;
    const size_t lists = (size_t)rows * cut.pieces;
    Args a;
    a.err = pool->err;
    a.logits = logits;
    a.stride = row_stride;
    a.vocab = vocab;
    a.k = k;
    a.cut = cut;
    a.keys = static_cast<uint64_t *>(pool->ws);
    a.sum = reinterpret_cast<double *>(a.keys + lists * k);
    a.top = reinterpret_cast<float *>(a.sum + lists);
    a.scores = scores;
    a.tickets = pool->tickets;
    a.tokens = tokens;
    a.parents = parents;
    a.out = out_scores;
    LaunchScope ls(pool, kDecode, s);
    const dim3 grid((unsigned)cut.pieces, (unsigned)batch, (unsigned)beams);
    cudaError_t e = elem == 4 ? launch_pdl(beam_select_kernel<float>, grid, dim3(kThreads), sizeof(Shared), s, a)
                              : launch_pdl(beam_select_kernel<__nv_bfloat16>, grid, dim3(kThreads), sizeof(Shared), s, a);
    ls.done();
    if (e != cudaSuccess) return cuda_fail(e, "paged_beam_select launch");
    return PKV_OK;
}
