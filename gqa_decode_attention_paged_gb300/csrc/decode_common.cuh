// What the decode kernels share: the stream of (sequence, KV head, block) items
// cut into equal slices, and the warp-level tensor-core and shared-memory
// helpers.
#pragma once

#include "pkv_internal.cuh"

namespace pkv {

// Exclusive prefix sum of block counts per sequence (after the first `skip`
// table entries) into ps[0..batch], the clamped lengths into cl and each
// sequence's first table entry into rb (each if not null); range errors go
// to *err when err is not null.  A sequence's table row is W entries from
// b * W (dense form) or entries indptr[b] .. indptr[b+1] of n_indices (CSR
// form; a row outside that range counts as empty).  warp_tot is scratch for
// NW ints.  The decode and merge kernels both derive their work from it.
template <int NW>
__device__ void scan_blocks(const int32_t *lens, int batch, int W, const int32_t *indptr, int64_t n_indices,
                            int skip, unsigned *err, int32_t *ps, int32_t *cl, int32_t *rb, int *warp_tot)
{
    constexpr int NT = NW * 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int carry = 0;
    for (int base = 0; base < batch; base += NT) {
        const int b = base + tid;
        int n = 0;
        if (b < batch) {
            int c = lens[b];
            int width = W, row = b * W;
            if (indptr) {
                const int32_t lo = indptr[b], hi = indptr[b + 1];
                const bool ok = lo >= 0 && lo <= hi && (int64_t)hi <= n_indices;
                if (!ok && err) atomicOr(err, PKV_DEVERR_BLOCK_RANGE);
                width = ok ? hi - lo : 0;
                row = ok ? lo : 0;
            }
            if (rb) rb[b] = row;
            const int cmax = width > (INT32_MAX / kBlockSize) ? INT32_MAX : width * kBlockSize;
            if (c < 0 || c > cmax) {
                if (err) atomicOr(err, PKV_DEVERR_CTX_RANGE);
                c = c < 0 ? 0 : cmax;
            }
            if (c < skip * kBlockSize) {  // cascade: every sequence holds the whole prefix
                if (err) atomicOr(err, PKV_DEVERR_CTX_RANGE);
                c = skip * kBlockSize;
            }
            if (cl) cl[b] = c;
            n = (c + kBlockSize - 1) / kBlockSize - skip;  // blocks after the shared prefix
        }
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_tot[warp] = x;
        __syncthreads();
        int before = 0, tot = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const int t = warp_tot[w];
            before += (w < warp) ? t : 0;
            tot += t;
        }
        if (b < batch) ps[b] = carry + before + x - n;
        carry += tot;
        __syncthreads();
    }
    if (tid == 0) ps[batch] = carry;
    __syncthreads();
}

// The stream: item f (0 <= f < total = n_kv * ps[batch]) is block j of head g
// of sequence b with f = n_kv * ps[b] + g * nblk_b + j.  Slice s covers items
// [s * share, (s + 1) * share); warp `me` of the grid takes slices me,
// me + n_warps, ...
struct Stream {
    const int32_t *ps;
    int batch, n_kv, total, share, n_slices, n_warps;
};

// One piece: blocks [j0, j1) of (b, g), starting at stream item f, in slice.
struct Piece {
    int b, g, j0, j1, nblk, f, slice;
};

__device__ __forceinline__ Piece locate(const Stream &st, int f, int slice)
{
    Piece p;
    int lo = 0, hi = st.batch - 1;  // largest b with n_kv * ps[b] <= f
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (st.n_kv * st.ps[mid] <= f) lo = mid; else hi = mid - 1;
    }
    p.b = lo;
    p.nblk = st.ps[lo + 1] - st.ps[lo];
    const int r = f - st.n_kv * st.ps[lo];
    p.g = r / p.nblk;
    p.j0 = r - p.g * p.nblk;
    const int slice_end = min(st.total, (slice + 1) * st.share);
    p.j1 = min(p.nblk, p.j0 + (slice_end - f));
    p.f = f;
    p.slice = slice;
    return p;
}

// The piece after p in this warp's walk.
__device__ __forceinline__ bool next_piece(const Stream &st, Piece &p)
{
    int f = p.f + (p.j1 - p.j0);
    int slice = p.slice;
    if (f >= min(st.total, (slice + 1) * st.share)) {
        slice += st.n_warps;
        if (slice >= st.n_slices) return false;
        f = slice * st.share;
    }
    p = locate(st, f, slice);
    return true;
}

__device__ __forceinline__ bool first_piece(const Stream &st, int me, Piece &p)
{
    if (me >= st.n_slices) return false;
    p = locate(st, me * st.share, me);
    return true;
}

// The producer walks the warp's blocks in segments of at most 32 consecutive
// blocks j .. j+n-1 of one piece.  One coalesced load fetches a segment's
// block-table entries (lane k holds block j+k's), one segment ahead of use,
// so no table read sits in front of a copy.
struct Seg {
    Piece p;
    int j, n;
    bool live;
};

__device__ __forceinline__ void seg_first(Seg &s, const Stream &st, int me)
{
    s.live = first_piece(st, me, s.p);
    s.j = s.live ? s.p.j0 : 0;
    s.n = s.live ? min(32, s.p.j1 - s.j) : 0;
}

__device__ __forceinline__ void seg_next(Seg &s, const Stream &st)
{
    if (!s.live) return;
    s.j += s.n;
    if (s.j >= s.p.j1) {
        s.live = next_piece(st, s.p);
        if (!s.live) {
            s.n = 0;
            return;
        }
        s.j = s.p.j0;
    }
    s.n = min(32, s.p.j1 - s.j);
}

// ---------------------------------------------------------------------------
// Warp-level tensor-core helpers (16x8x16 MMA, bf16 or f16 in, fp32 out)
// ---------------------------------------------------------------------------

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2^x with the MUFU approximation (relative error about 2^-22; results below
// 2^-126 flush to 0, 2^-inf = 0 and 2^0 = 1).  The decode softmax's weights use it.
__device__ __forceinline__ float ex2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void prefetch_l2(const void *p)
{
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Transpose an 8x8 matrix of 16-bit values held one row-pair per thread.
__device__ __forceinline__ uint32_t movm_t(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel)
{
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

// Four E4M3 bytes -> two f16x2 words (bytes 0,1 -> lo; bytes 2,3 -> hi); exact.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t x, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (F16) {
        __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    }
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

// Byte offset inside a TMA box region (aligned to its swizzle atom) after the
// box's swizzle: 16-byte chunk index XOR the 128-byte line index (mod 8) for
// 128-byte rows, XOR (line index mod 4) for 64-byte rows.
template <int BOXB>
__device__ __forceinline__ uint32_t swz(uint32_t off)
{
    if constexpr (BOXB == 128) return off ^ ((off >> 3) & 0x70u);
    else if constexpr (BOXB == 64) return off ^ ((off >> 3) & 0x30u);
    else return off ^ ((off >> 3) & 0x10u);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}


}  // namespace pkv
