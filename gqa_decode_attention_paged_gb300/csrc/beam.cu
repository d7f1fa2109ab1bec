// Beam search's selection over beams and vocabulary.
//
// Mathematics.  Candidate (beam j, token t) of a search is worth
//   v = score_j + x_jt - lse_j,   lse_j = log sum_t exp x_jt;
// the k greatest are selected, equal ones by the lower j * vocab + t.  Within
// a row v grows with x, so a row's candidates are its k greatest logits, and
// only those need v.
//
// What bounds it: HBM, the logits read once; close behind it the exponentials
// (one per logit, 16 an SM and cycle).  Two launches: a scan of the rows, cut
// into slices so that every SM has work, leaves each slice's maximum, sum of
// exponentials and k greatest logits; a merge of each search's lists.
//
// Selecting while scanning.  From a slice's first part (kVecs vectors of 16
// bytes per thread) the threads' greatest logits, reduced to 4 k groups or more,
// give a bar: the k-th greatest group maximum, which at least k logits reach.
// Those that do belong to k groups, so they fit the buffer whatever the data.
// The warps then read the rest each for itself, without barriers, and add what
// is above the bar: k (n / n_1 - 1) logits where they come in any order.  Only
// where they rise along the row can the buffer run over; the slice is then read
// again in parts, each of which raises the bar first.  Keys (logit as an ordered
// integer, then the lower index) are unique, so ties need no care and results do
// not depend on the order of arrival.
//
// A row may begin anywhere.  Which thread adds which logits must not depend on
// that, or two beams with equal logits would get sums that differ in the last
// place, and equal continuations would not go to the lower beam.  So a lane
// takes the N elements from a multiple of N of the row on, out of two aligned
// vectors: its own and the next lane's.  The last lane of a warp only passes
// its vector on.
//
// Accuracy.  Candidates of different beams may lie arbitrarily close, so what
// decides between them is held in more than 32 bits: the exponentials are
// 32-bit (of x - m, exact near the maximum, where they count), a thread's sum
// too, all further sums are 64-bit integers (2^-40 of the largest term), and
// the logarithm and v are doubles.
#include <algorithm>
#include <climits>
#include <math.h>

#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;                         // 16-byte vectors of a thread in a part
constexpr int kLanes = 31;                       // lanes of a warp that have logits
constexpr int kRunVecs = kWarps * kLanes;        // a vector each: the unit in which rows are cut
constexpr int kMaxK = 64, kMaxBeams = 64;
constexpr int kCap = 5120;                       // keys the buffer holds: a part's 4096 at most, k kept ones, some more
constexpr int kMaxLists = 1024;                  // (beam, slice) lists of a search
constexpr int kMergeThreads = 256;
constexpr int kMergeKeys = 4096;                 // keys of a search that the merge holds in shared memory

struct ScanArgs {
    const void *logits;
    int64_t stride;  // elements between rows
    int vocab, k, slices;
    uint64_t *keys;  // [rows][slices][k], greatest first, 0: none
    float *top;      // [rows][slices] maximum
    double *sum;     // [rows][slices] sum of exp(x - maximum); NaN where the slice holds a NaN or +infinity
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
    uint64_t buf[kCap];
    uint64_t group[256];
    uint64_t bar;      // keys below it are not among the k greatest
    uint64_t sums[kWarps];
    float tops[kWarps];
    int n;             // keys in buf (those past kCap are not there)
};

__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// Raises sh.bar to the k-th greatest of the groups' greatest keys (of `mine`, 0: none; 16 p groups of 32 / p
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

// A row of logits, as one warp reads it: run r is kLanes vectors of every warp, a vector a lane.
template <typename T>
struct Row {
    using El = Elems<T>;
    static constexpr int N = El::N;
    const T *x;
    int vocab, lead;  // elements before the row in its first aligned vector
    int lane, warp;

    // index of this lane's first element of run r
    __device__ __forceinline__ int first(int r) const { return ((r * kWarps + warp) * kLanes + lane) * N; }
    // the aligned vector in which it is
    __device__ __forceinline__ uint4 load(int r) const
    {
        const int i = first(r) - lead;
        if (i >= 0 && i <= vocab - N) return ldg_nc_v4(x + i);
        uint32_t w[4] = {El::kLow, El::kLow, El::kLow, El::kLow};  // the row's ends
        if (i > -N && i < vocab) {
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
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // this lane's elements, from its vector and the next lane's
    __device__ __forceinline__ uint4 line_up(const uint4 &r) const
    {
        uint32_t w[8] = {r.x, r.y, r.z, r.w};
        if (lead) {
            const int words = lead * (int)sizeof(T) / 4;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[4 + i] = __shfl_down_sync(kFull, w[i], 1);
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
        }
        const bool on = lane < kLanes;
        return make_uint4(on ? w[0] : El::kLow, on ? w[1] : El::kLow, on ? w[2] : El::kLow, on ? w[3] : El::kLow);
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

// A thread's greatest logit so far and the sum of exp(x - m).
struct Sum {
    float m = -INFINITY, s = 0.0f;
    // kVecs vectors with the greatest logit top
    template <typename T>
    __device__ __forceinline__ void add(const uint4 (&v)[kVecs], float top)
    {
        constexpr int N = Elems<T>::N;
        if (top > m) {
            s = m == -INFINITY ? s : s * ex2((m - top) * kLog2e);
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
        s += part.x + part.y;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) beam_scan_kernel(const __grid_constant__ ScanArgs a)
{
    using El = Elems<T>;
    constexpr int N = El::N;
    __shared__ Shared sh;
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slice = blockIdx.x;
    const int64_t row = (int64_t)blockIdx.y * gridDim.z + blockIdx.z;  // (search, beam)
    Row<T> rw;
    rw.x = static_cast<const T *>(a.logits) + row * a.stride;
    rw.vocab = a.vocab;
    rw.lead = (int)(((uintptr_t)rw.x & 15u) / sizeof(T));
    rw.lane = lane;
    rw.warp = warp;
    const int runs = (a.vocab + kRunVecs * N - 1) / (kRunVecs * N);
    const int r0 = (int)((int64_t)runs * slice / a.slices), r1 = (int)((int64_t)runs * (slice + 1) / a.slices);
    const int k = a.k;
    const int p = k <= 4 ? 1 : k <= 8 ? 2 : k <= 16 ? 4 : k <= 32 ? 8 : 16;  // groups of a warp
    if (tid == 0) {
        sh.n = 0;
        sh.bar = 0;
    }
    const uint4 none = make_uint4(El::kLow, El::kLow, El::kLow, El::kLow);
    auto load = [&](int r, uint4 (&v)[kVecs]) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = r + i < r1 ? rw.load(r + i) : none;
    };
    auto line_up = [&](uint4 (&v)[kVecs]) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = rw.line_up(v[i]);
    };
    auto greatest = [&](const uint4 (&v)[kVecs]) -> float {
        static_assert(kVecs == 4, "");
        return fmaxf(fmaxf(greatest_of<T>(v[0]), greatest_of<T>(v[1])), fmaxf(greatest_of<T>(v[2]), greatest_of<T>(v[3])));
    };
    // the key of a thread's greatest logit: of equal ones the first
    auto key_at = [&](const uint4 (&v)[kVecs], int r, float top) -> uint64_t {
        if (!(top > -INFINITY)) return 0;
        int at = 0;
#pragma unroll
        for (int i = kVecs - 1; i >= 0; --i) {
            float x[N];
            El::widen(v[i], x);
#pragma unroll
            for (int e = N - 1; e >= 0; --e) at = x[e] == top ? i * (kRunVecs * N) + e : at;
        }
        return key_of(top, rw.first(r) + at);
    };
    // adds this thread's logits that reach the bar to the buffer
    auto add_keys = [&](const uint4 (&v)[kVecs], int r, uint64_t bar) {
#pragma unroll 1
        for (int i = 0; i < kVecs; ++i) {
            const uint4 w = i == 0 ? v[0] : i == 1 ? v[1] : i == 2 ? v[2] : v[3];
            const float top = greatest_of<T>(w);
            if (!(top > -INFINITY) || (bar && top < logit_of(bar))) continue;
            float x[N];
            El::widen(w, x);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if (!(x[e] > -INFINITY)) continue;
                const uint64_t key = key_of(x[e], rw.first(r + i) + e);
                if (key < bar) continue;
                const int at = atomicAdd(&sh.n, 1);
                if (at < kCap) sh.buf[at] = key;
            }
        }
    };
    Sum sum;
    uint4 cur[kVecs], nxt[kVecs];
    load(r0, cur);
    load(r0 + kVecs, nxt);
    line_up(cur);
    float top = greatest(cur);
    __syncthreads();  // (the bar and the count are set)
    raise_bar(sh, key_at(cur, r0, top), k, p);
    uint64_t bar = sh.bar;
    add_keys(cur, r0, bar);
    sum.add<T>(cur, top);
    // ---- the rest of the slice, every warp for itself ----
    const float high = bar ? logit_of(bar) : -INFINITY;
    for (int r = r0 + kVecs; r < r1; r += kVecs) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) cur[i] = nxt[i];
        load(r + kVecs, nxt);
        line_up(cur);
        top = greatest(cur);
        if (top > high) add_keys(cur, r, bar);  // (an equal one has a greater index than the bar's)
        sum.add<T>(cur, top);
    }
    // ---- the slice's maximum and sum ----
    float M = sum.m;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    if (lane == 0) sh.tops[warp] = M;
    const bool bad = __syncthreads_or(!(sum.s < INFINITY));  // (the sum of a NaN or an infinite logit is NaN)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh.tops[w]);
    uint64_t f = 0;  // this thread's sum in units of 2^-40
    if (!bad && sum.m > -INFINITY) f = __float2ull_rn(sum.s * ex2((sum.m - M) * kLog2e) * 0x1p40f);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) f += __shfl_xor_sync(kFull, f, o);
    if (lane == 0) sh.sums[warp] = f;
    int n = sh.n;  // (no keys are added any more)
    __syncthreads();
    if (n > kCap) {  // the buffer ran over: the slice again, part by part
        if (tid == 0) {
            sh.n = 0;
            sh.bar = 0;
        }
        __syncthreads();
        for (int r = r0; r < r1; r += kVecs) {
            const int have = sh.n;
            load(r, cur);
            line_up(cur);
            raise_bar(sh, key_at(cur, r, greatest(cur)), k, p);
            if (have + 4096 > kCap) thin_out(sh, have, k, p, kMaxK);
            add_keys(cur, r, sh.bar);
            __syncthreads();
        }
        n = sh.n;
        __syncthreads();
    }
    n = thin_out(sh, n, k, p, 256);
    const int64_t list = row * a.slices + slice;
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
}

struct MergeArgs {
    const uint64_t *keys;
    const float *top;
    const double *sum;
    const float *scores;  // [batch][beams]
    int beams, slices, k;
    int32_t *tokens, *parents;  // [batch][k]
    float *out;                 // [batch][k]
    unsigned *err;
};

// A continuation: its worth as an ordered integer (0: none), its beam and its key.  Equal worths go to the lower
// beam, then to the greater key (doubles may round a beam's different logits to one worth).
struct Best {
    uint64_t value, key;
    int beam;
    __device__ __forceinline__ bool before(const Best &y) const
    {
        return value != y.value ? value > y.value : beam != y.beam ? beam < y.beam : key > y.key;
    }
};

__device__ __forceinline__ uint64_t warp_max(uint64_t x, bool on)
{
    const uint32_t hi = __reduce_max_sync(kFull, on ? (uint32_t)(x >> 32) : 0u);
    const uint32_t lo = __reduce_max_sync(kFull, on && (uint32_t)(x >> 32) == hi ? (uint32_t)x : 0u);
    return ((uint64_t)hi << 32) | lo;
}

// The first of a warp's.
__device__ __forceinline__ Best warp_best(const Best &x)
{
    const uint64_t value = warp_max(x.value, true);
    unsigned on = __ballot_sync(kFull, x.value == value);
    if (on & (on - 1)) {  // the same for all lanes
        const int beam = __reduce_min_sync(kFull, x.value == value ? x.beam : INT_MAX);
        const bool mine = x.value == value && x.beam == beam;
        const uint64_t key = warp_max(x.key, mine);
        on = __ballot_sync(kFull, mine && x.key == key);
    }
    const int l = __ffs(on) - 1;
    return {value, __shfl_sync(kFull, x.key, l), __shfl_sync(kFull, x.beam, l)};
}

// One search: its beams' log-sums, then k times the best of the lists' heads.
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const __grid_constant__ MergeArgs a)
{
    __shared__ double shift[kMaxBeams];  // score - log of the sum of exp(x - m); NaN: no candidates
    __shared__ float highest[kMaxBeams]; // m: v = (x - m) + shift, in which large logits cost nothing
    __shared__ uint64_t held[kMergeKeys];
    __shared__ uint8_t at[kMaxLists];    // keys of a list that are taken
    __shared__ Best bests[2][kMergeThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t item = blockIdx.x;
    const int lists = a.beams * a.slices, total = lists * a.k;
    const uint64_t *keys = a.keys + item * total;
    const bool hold = total <= kMergeKeys;
    if (hold)
        for (int i = tid; i < total; i += kMergeThreads) held[i] = keys[i];
    for (int i = tid; i < lists; i += kMergeThreads) at[i] = 0;
    for (int j = warp; j < a.beams; j += kMergeThreads / 32) {  // a warp a beam, a lane a slice
        const int64_t l0 = (item * a.beams + j) * a.slices;
        float M = -INFINITY;
        for (int i = lane; i < a.slices; i += 32) M = fmaxf(M, a.top[l0 + i]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
        double s = 0.0;
        for (int i = lane; i < a.slices; i += 32) {
            const float t = a.top[l0 + i];
            const double x = a.sum[l0 + i];  // (of an infinite maximum NaN)
            s += t == M || x != x ? x : t == -INFINITY ? 0.0 : x * exp((double)t - (double)M);
        }
        for (int o = 16; o >= 1; o >>= 1)
            if (o < a.slices) s += __shfl_xor_sync(kFull, s, o);  // (lanes past the slices hold 0)
        if (lane) continue;
        const float sc = a.scores[item * a.beams + j];
        const bool odd = sc != -INFINITY && (s != s || sc != sc || sc == INFINITY);
        if (odd) atomicOr(a.err, PKV_DEVERR_NAN);
        shift[j] = odd || sc == -INFINITY || M == -INFINITY ? (double)NAN : (double)sc - log(s);
        highest[j] = M;
    }
    __syncthreads();
    constexpr Best kNone = {0, 0, INT_MAX};
    auto head = [&](int l) -> Best {  // of a list
        const int n = at[l], j = l / a.slices;
        if (n >= a.k) return kNone;
        const uint64_t key = hold ? held[l * a.k + n] : keys[(int64_t)l * a.k + n];
        const double v = ((double)logit_of(key) - (double)highest[j]) + shift[j];
        if (!key || v != v) return kNone;
        const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
        return {u ^ ((u >> 63) ? ~0ull : 1ull << 63), key, j};
    };
    const bool alone = lists <= 32;  // one warp has all lists
    if (alone && warp) return;
    Best mine;
    int from = 0;
    auto look = [&]() {
        mine = kNone;
        for (int l = tid; l < lists; l += kMergeThreads) {
            const Best x = head(l);
            if (x.before(mine)) {
                mine = x;
                from = l;
            }
        }
    };
    look();
    for (int i = 0; i < a.k; ++i) {
        Best w = warp_best(mine);
        if (!alone) {
            if (lane == 0) bests[i & 1][warp] = w;
            __syncthreads();
            w = warp_best(lane < kMergeThreads / 32 ? bests[i & 1][lane] : kNone);
        }
        const int64_t o = item * a.k + i;
        if (w.value == 0) {  // no candidate is left
            if (tid == 0) {
                a.tokens[o] = a.parents[o] = -1;
                a.out[o] = -INFINITY;
            }
        } else if (mine.beam == w.beam && mine.key == w.key) {
            const uint64_t u = w.value ^ ((w.value >> 63) ? 1ull << 63 : ~0ull);
            a.tokens[o] = index_of(w.key);
            a.parents[o] = w.beam;
            a.out[o] = (float)__longlong_as_double((long long)u);
            ++at[from];
            look();
        }
    }
}

// Slices of a row: enough for two blocks on every SM, no more than the row has parts, nor than the merge takes.
int slices_of(const pkv_pool *pool, int64_t rows, int beams, int vocab, int elem)
{
    const int64_t part = (int64_t)kRunVecs * kVecs * (16 / elem);
    const int64_t parts = (vocab + part - 1) / part;
    const int64_t want = std::max<int64_t>(1, 2 * (int64_t)pool->num_sms / std::max<int64_t>(1, rows));
    return (int)std::max<int64_t>(1, std::min({want, parts, (int64_t)(kMaxLists / beams)}));
}

size_t beam_bytes(int64_t rows, int slices, int k) { return (size_t)rows * slices * (8 * (size_t)k + 16); }

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

bool overlap(const void *x, size_t xn, const void *y, size_t yn)
{
    return (uintptr_t)x < (uintptr_t)y + yn && (uintptr_t)y < (uintptr_t)x + xn;
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
    for (int b = 1; b <= batch; ++b)  // (calls of fewer rows have more slices)
        for (int elem : {2, 4}) {
            const int64_t rows = (int64_t)b * beams;
            most = std::max(most, beam_bytes(rows, slices_of(pool, rows, beams, vocab, elem), k));
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
    const int slices = slices_of(pool, rows, beams, vocab, elem);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = ensure_workspace(pool, beam_bytes(rows, slices, k), s, who);
    if (st != PKV_OK) return st;
    const size_t lists = (size_t)rows * slices;
    ScanArgs a;
    a.logits = logits;
    a.stride = row_stride;
    a.vocab = vocab;
    a.k = k;
    a.slices = slices;
    a.keys = static_cast<uint64_t *>(pool->ws);
    a.sum = reinterpret_cast<double *>(a.keys + lists * k);
    a.top = reinterpret_cast<float *>(a.sum + lists);
    {
        LaunchScope ls(pool, kDecode, s);
        const dim3 grid((unsigned)slices, (unsigned)batch, (unsigned)beams);
        cudaError_t e = elem == 4 ? launch_pdl(beam_scan_kernel<float>, grid, dim3(kThreads), 0, s, a)
                                  : launch_pdl(beam_scan_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, a);
        ls.done();
        if (e != cudaSuccess) return cuda_fail(e, "paged_beam_select scan launch");
    }
    MergeArgs m;
    m.keys = a.keys;
    m.top = a.top;
    m.sum = a.sum;
    m.scores = scores;
    m.beams = beams;
    m.slices = slices;
    m.k = k;
    m.tokens = tokens;
    m.parents = parents;
    m.out = out_scores;
    m.err = pool->err;
    LaunchScope ls(pool, kMerge, s);
    cudaError_t e = launch_pdl(beam_merge_kernel, dim3((unsigned)batch), dim3(kMergeThreads), 0, s, m);
    ls.done();
    if (e != cudaSuccess) return cuda_fail(e, "paged_beam_select merge launch");
    return PKV_OK;
}
