// Rotary cache write: rotate each new token's queries and keys by its
// position and write the rotated key row and the value row into the pool,
// quantised on the way in as paged_kv_append quantises.
//
// Mathematics.  Pair i of a head (two of its first rot_dim channels) is a
// point in the plane, turned by angle_i = position[axis_i] * inv_freq[i]:
//   (a, b) -> (a cos - b sin, b cos + a sin).
// Positions are whole numbers, so only the fraction of a turn that inv_freq
// makes per position matters: the host stores turn_i = frac(inv_freq[i] /
// 2 pi) as a 64-bit fixed-point fraction (turn_fraction), the kernel multiplies
// it by the position modulo 2^64 (exact, whatever the position) and takes sine
// and cosine of the top 32 bits (turn_of).  The angle is thus off by at most
// 2^-34 of a turn from the fraction's rounding, at the farthest position, and
// 2^-33 from the top bits': below 2^-32 at every position, where a 32-bit
// product would be off by 2^-24 * angle (0.004 radians at 65536), without
// 64-bit floating point in the kernel.
// The rotation runs in fp32 and is rounded once: to bf16 (queries, bf16
// pools), to E4M3 or to the 4-bit code.
//
// What bounds it: HBM (about 0.7 operations a byte).  One warp takes one
// token (or, when there are few tokens, one share of its heads): D / 16 lanes
// per head row, each holding two 16-byte chunks that make 8 whole pairs, so a
// rotation needs no exchange between lanes; the 32 / (D / 16) lanes that hold
// the same pairs of different heads compute 8 sines and cosines between them
// and swap them by shuffles, once for all heads of the token.
// 20321 image tokens (32 query, 8 KV heads of 128, E4M3): 82 us, 84 % of the
// copy rate; a decode step's 64 tokens: 6.2 us, the latency of a launch and of
// two dependent loads.
#include "pkv_internal.cuh"
#include "turn.cuh"

#include <math.h>

#include <algorithm>
#include <new>

// Host handle: what rotates (see pkv_rope_create).
struct pkv_rope {
    int rot_dim = 0, interleaved = 0, n_axes = 0;
    uint64_t turn[64] = {};  // per pair: frac(inv_freq / 2 pi) * 2^64
    uint8_t axis[64] = {};
};

namespace pkv {
namespace {

constexpr int kRopeWarps = 2;  // warps per CTA (2: 81 us, 4: 82, at the tokens below)
// What was tried is quoted for 20321 image tokens to an E4M3 pool (459 MB: 69 us at the copy rate), and for 9625
// tokens written to a 4-bit pool and read back (42 in all, 33 of them the write).
// Head rows a lane has in flight: 1: 94 us, 2: 82, 3: 96; 4-bit pools 1: 43, 2: 45, 3: 45.
constexpr int unroll_of(int kv) { return kv == PKV_INT4 ? 1 : 2; }
// CTAs an SM has room for, which bounds the registers: 20 warps 82 us, 24: 88; 4-bit pools 47 and 45.
constexpr int ctas_of(int kv) { return kv == PKV_INT4 ? 12 : 10; }

struct RopeArgs {
    uint64_t turn[64];
    uint8_t axis[64];
    int rot_dim;
    const __nv_bfloat16 *q, *k, *v;  // token rows at q_stride, k_stride, v_stride elements
    __nv_bfloat16 *q_out;
    int64_t q_stride, k_stride, v_stride, qo_stride;
    int n_q, n_kv;
    const int32_t *positions;  // [n_axes][n_tokens]
    const int64_t *slots;
    int64_t n_tokens;
    int splits;                // warps that share a token's heads
    uint8_t *pool;
    int64_t num_blocks;
    const float *scales;       // FP8: [2 * n_kv]
    const float *k_params;     // 4-bit: [2][n_kv][D]
    unsigned *err;
};

// 4-bit code of x: clamp(rint((x - z) / s), 0, 15), each step correctly rounded in fp32, NaN to 0.  `r` is
// 1 / s to a few units of its last place, or NaN: the product with it is off by less than 2^-17 where the code is
// not clamped, so the correctly rounded quotient is needed only next to a border between two codes (or
// where the product is not finite); everywhere else both round to the same code.
__device__ __forceinline__ uint32_t code4(float x, float s, float z, float r)
{
    const float d = __fsub_rn(x, z);
    float q = d * r, c = rintf(q);
    if (!(fabsf(q - c) < 0.49998f)) c = rintf(__fdiv_rn(d, s));
    return c >= 0.0f ? (uint32_t)fminf(c, 15.0f) : 0u;
}

__device__ __forceinline__ float rcp_approx(float s)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return r;
}

// Codes of 8 channels whose scales and zero points lie one after the other (16-byte aligned).
__device__ __forceinline__ uint32_t key_codes(const float *x, const float *ks, const float *kz)
{
    const float4 s[2] = {__ldg(reinterpret_cast<const float4 *>(ks)), __ldg(reinterpret_cast<const float4 *>(ks) + 1)};
    const float4 z[2] = {__ldg(reinterpret_cast<const float4 *>(kz)), __ldg(reinterpret_cast<const float4 *>(kz) + 1)};
    const float sv[8] = {s[0].x, s[0].y, s[0].z, s[0].w, s[1].x, s[1].y, s[1].z, s[1].w};
    const float zv[8] = {z[0].x, z[0].y, z[0].z, z[0].w, z[1].x, z[1].y, z[1].z, z[1].w};
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)  // (from 2^126 on 1 / s is below fp32's normal range, and NaN asks for the quotient)
        w |= code4(x[i], sv[i], zv[i], sv[i] < 0x1p126f ? rcp_approx(sv[i]) : __int_as_float(0x7fffffff)) << (4 * i);
    return w;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint4 pack_bf16(const float *x)
{
    return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}

// E4M3 codes of x / s, the quotient correctly rounded in fp32, from r = 1 / s to two units of its last place.  The
// product with r is off by less than 8 units; in E4M3's normal range that leaves the code as it is unless the 20 bits
// that the rounding drops are that close to a half.  Only there, and below that range or where r is not in fp32's, is
// the quotient itself needed (dividing always took 90 us of 20321 image tokens, this 82).
__device__ __forceinline__ uint2 pack_e4m3(const float *x, float s, float r)
{
    float y[8];
    bool close = !(s > 0x1p-100f && s < 0x1p100f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = x[i] * r;
        const uint32_t dropped = __float_as_uint(y[i]) & 0xfffffu;
        close |= dropped - 0x7fff8u <= 0x10u || fabsf(y[i]) < 0x1p-6f;
    }
    if (close) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], s);
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t e = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i], y[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        w[i >> 1] = (i & 1) ? w[i >> 1] | (e << 16) : e;
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void widen(uint4 r, float *x)
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf16x2_to_f32x2(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <int D, int KV, bool INTER>
__global__ void __launch_bounds__(kRopeWarps * 32, ctas_of(KV)) rope_append_kernel(const __grid_constant__ RopeArgs a)
{
    constexpr int kUnroll = unroll_of(KV);
    constexpr int LPR = D / 16;     // lanes per head row
    constexpr int RPW = 32 / LPR;   // head rows per warp and step
    constexpr int PPL = 8 / RPW;    // pairs whose sine and cosine a lane computes
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int j = lane % LPR, r = lane / LPR;
    const int64_t w = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    const int64_t t = w / a.splits;
    const int part = (int)(w - t * a.splits);
    if (t >= a.n_tokens) return;  // the whole warp

    // This lane's two chunks of 8 channels: pairs (i, i + rot_dim / 2), or adjacent channels
    // (interleaved pairs, and the channels past rot_dim, which are copied).
    const int half = a.rot_dim / 16;  // chunks of one half of the rotated channels = lanes that rotate
    const bool turns = j < half;
    const int c0 = (INTER || !turns) ? 2 * j : j, c1 = (INTER || !turns) ? 2 * j + 1 : j + half;

    const int64_t slot = a.slots[t];
    const int rows = a.n_q + 2 * a.n_kv;  // head rows of a token: queries, keys, values
    // row `row` of the token: where it is read
    auto source = [&](int row) -> const __nv_bfloat16 * {
        if (row < a.n_q) return a.q + t * a.q_stride + (int64_t)row * D;
        row -= a.n_q;
        if (row < a.n_kv) return a.k + t * a.k_stride + (int64_t)row * D;
        return a.v + t * a.v_stride + (int64_t)(row - a.n_kv) * D;
    };
    const int step = a.splits * RPW;
    uint4 x0[kUnroll], x1[kUnroll];
    auto fetch = [&](int u, int row) {
        if (row < rows) {
            const __nv_bfloat16 *src = source(row);
            x0[u] = *reinterpret_cast<const uint4 *>(src + 8 * c0);
            x1[u] = *reinterpret_cast<const uint4 *>(src + 8 * c1);
        }
    };
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        fetch(u, part * RPW + r + u * step);  // in flight while the sines and cosines are computed

    // pairs 8 j .. 8 j + 7 are this lane's; lane r of the RPW lanes with the same j computes PPL of them
    float cs[8], sn[8];
    {
        float c[PPL], s[PPL];
#pragma unroll
        for (int i = 0; i < PPL; ++i) {
            c[i] = 1.0f;
            s[i] = 0.0f;
            if (turns) {
                const int pair = 8 * j + r * PPL + i;
                const int64_t pos = a.positions[(int64_t)a.axis[pair] * a.n_tokens + t];
                const uint64_t frac = a.turn[pair] * (uint64_t)pos;  // fraction of a turn, modulo 2^64
                turn_of((uint32_t)((frac + 0x80000000ull) >> 32), s[i], c[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int src = (i / PPL) * LPR + j;
            cs[i] = __shfl_sync(kFull, c[i % PPL], src);
            sn[i] = __shfl_sync(kFull, s[i % PPL], src);
        }
    }

    const int64_t slots = a.num_blocks * kBlockSize;
    bool keep = slot >= 0;
    if (slot >= slots) {
        keep = false;
        if (lane == 0) atomicOr(a.err, PKV_DEVERR_SLOT_RANGE);
    }
    const int64_t blk = slot / kBlockSize;
    const int off = (int)(slot - blk * kBlockSize);

    // every lane of the warp makes the same number of steps (the 4-bit value rows shuffle)
    for (int base = part * RPW; base < rows; base += kUnroll * step) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int row0 = base + u * step;
            if (row0 >= rows) break;
            const int row = row0 + r;
            const bool live = row < rows;
            const int kvrow = row - a.n_q;  // < 0: a query; < n_kv: a key; else a value
            const bool is_v = kvrow >= a.n_kv;
            float y0[8], y1[8];
            const uint4 r0 = x0[u], r1 = x1[u];
            fetch(u, row + kUnroll * step);  // the place is free: the row kUnroll steps on
            if (live) {
                float lo[8], hi[8];
                widen(r0, lo);
                widen(r1, hi);
                if (!is_v && turns) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        // pair i: (lo[i], hi[i]), or adjacent channels of the two chunks
                        const float p = INTER ? (i < 4 ? lo[2 * (i & 3)] : hi[2 * (i & 3)]) : lo[i];
                        const float s = INTER ? (i < 4 ? lo[2 * (i & 3) + 1] : hi[2 * (i & 3) + 1]) : hi[i];
                        const float pr = fmaf(p, cs[i], -s * sn[i]), sr = fmaf(s, cs[i], p * sn[i]);
                        if (INTER) {
                            if (i < 4) { y0[2 * (i & 3)] = pr; y0[2 * (i & 3) + 1] = sr; }
                            else { y1[2 * (i & 3)] = pr; y1[2 * (i & 3) + 1] = sr; }
                        } else {
                            y0[i] = pr;
                            y1[i] = sr;
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        y0[i] = lo[i];
                        y1[i] = hi[i];
                    }
                }
            }
            if (live && kvrow < 0) {
                __nv_bfloat16 *dst = a.q_out + t * a.qo_stride + (int64_t)row * D;
                *reinterpret_cast<uint4 *>(dst + 8 * c0) = pack_bf16(y0);
                *reinterpret_cast<uint4 *>(dst + 8 * c1) = pack_bf16(y1);
            }
            const int g = is_v ? kvrow - a.n_kv : kvrow;
            if constexpr (KV != PKV_INT4) {
                if (live && kvrow >= 0 && keep) {
                    constexpr int E = KV == PKV_BF16 ? 2 : 1;
                    uint8_t *dst = a.pool + (((blk * a.n_kv + g) * 2 + (is_v ? 1 : 0)) * kBlockSize + off) * (D * E);
                    if constexpr (KV == PKV_BF16) {
                        *reinterpret_cast<uint4 *>(dst + 16 * c0) = pack_bf16(y0);
                        *reinterpret_cast<uint4 *>(dst + 16 * c1) = pack_bf16(y1);
                    } else {
                        const float s = a.scales[is_v ? a.n_kv + g : g];
                        const float rs = rcp_approx(s);
                        *reinterpret_cast<uint2 *>(dst + 8 * c0) = pack_e4m3(y0, s, rs);
                        *reinterpret_cast<uint2 *>(dst + 8 * c1) = pack_e4m3(y1, s, rs);
                    }
                }
            } else {
                // a value row's min and max over its LPR lanes (rows of other kinds shuffle along)
                float mn = 0.0f, mx = 0.0f;
                if (live && is_v) {
                    mn = mx = y0[0];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        mn = fminf(mn, fminf(y0[i], y1[i]));
                        mx = fmaxf(mx, fmaxf(y0[i], y1[i]));
                    }
                }
#pragma unroll
                for (int o = 1; o < LPR; o <<= 1) {
                    mn = fminf(mn, __shfl_xor_sync(kFull, mn, o));
                    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
                }
                if (live && kvrow >= 0 && keep) {
                    uint8_t *entry = a.pool + (blk * a.n_kv + g) * i4_entry_bytes(D);
                    uint32_t w0 = 0, w1 = 0;
                    if (is_v) {
                        // (max - min) / 15 as one product with fp32(1/15): at most a step of the last place
                        // from paged_kv_append's quotient
                        float sc = __fmul_rn(__fsub_rn(mx, mn), 1.0f / 15.0f);
                        if (sc == 0.0f) sc = 1.0f;
                        const float z = __fadd_rn(mn, 0.0f);  // no negative zero
                        const float rc = rcp_approx(sc);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            w0 |= code4(y0[i], sc, z, rc) << (4 * i);
                            w1 |= code4(y1[i], sc, z, rc) << (4 * i);
                        }
                        if (j == 0)
                            *reinterpret_cast<float2 *>(entry + i4_params_offset(D) + off * 8) = make_float2(sc, z);
                        entry += i4_v_offset(D);
                    } else {
                        const float *ks = a.k_params + (int64_t)g * D, *kz = ks + (int64_t)a.n_kv * D;
                        w0 = key_codes(y0, ks + 8 * c0, kz + 8 * c0);
                        w1 = key_codes(y1, ks + 8 * c1, kz + 8 * c1);
                    }
                    *reinterpret_cast<uint32_t *>(entry + off * (D / 2) + 4 * c0) = w0;
                    *reinterpret_cast<uint32_t *>(entry + off * (D / 2) + 4 * c1) = w1;
                }
            }
        }
    }
}

template <int D, int KV, bool INTER>
cudaError_t launch_one(const RopeArgs &a, int64_t ctas, cudaStream_t s)
{
    return launch_pdl(rope_append_kernel<D, KV, INTER>, dim3((unsigned)ctas), dim3(kRopeWarps * 32), 0, s, a);
}

template <int D, int KV>
cudaError_t launch_inter(const RopeArgs &a, bool inter, int64_t ctas, cudaStream_t s)
{
    return inter ? launch_one<D, KV, true>(a, ctas, s) : launch_one<D, KV, false>(a, ctas, s);
}

template <int D>
cudaError_t launch_kv(const RopeArgs &a, int kv, bool inter, int64_t ctas, cudaStream_t s)
{
    if (kv == PKV_BF16) return launch_inter<D, PKV_BF16>(a, inter, ctas, s);
    if (kv == PKV_FP8_E4M3) return launch_inter<D, PKV_FP8_E4M3>(a, inter, ctas, s);
    return launch_inter<D, PKV_INT4>(a, inter, ctas, s);
}

// Whether two sets of n rows (width elements at stride, bf16) share an element.
bool rows_overlap(const void *pa, int64_t stride_a, int64_t wa, const void *pb, int64_t stride_b, int64_t wb, int64_t n)
{
    const int64_t a = (int64_t)((uintptr_t)pa / 2), b = (int64_t)((uintptr_t)pb / 2);
    if (a + (n - 1) * stride_a + wa <= b || b + (n - 1) * stride_b + wb <= a) return false;
    if (n > 1 && stride_a == stride_b) {  // rows of one wider array: compare the places inside a row
        const int64_t d = ((b - a) % stride_a + stride_a) % stride_a;
        return d < wa || d + wb > stride_a;
    }
    return true;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_rope_create(int32_t rot_dim, int32_t interleaved, int32_t n_axes, const double *inv_freq,
                                      const int32_t *pair_axis, pkv_rope **out)
{
    if (!out) return fail(PKV_EINVAL, "pkv_rope_create: out is NULL");
    *out = nullptr;
    if (rot_dim <= 0 || rot_dim % 16 || rot_dim > 128)
        return fail(PKV_EUNSUPPORTED, "pkv_rope_create: rot_dim %d unsupported (16, 32, ..., 128)", rot_dim);
    if (interleaved != 0 && interleaved != 1)
        return fail(PKV_EINVAL, "pkv_rope_create: interleaved must be 0 or 1, not %d", interleaved);
    if (n_axes < 1 || n_axes > 8) return fail(PKV_EINVAL, "pkv_rope_create: n_axes %d not in 1..8", n_axes);
    if (!inv_freq) return fail(PKV_EINVAL, "pkv_rope_create: inv_freq is NULL");
    for (int i = 0; i < rot_dim / 2; ++i) {
        if (!(fabs(inv_freq[i]) <= 1048576.0))
            return fail(PKV_EINVAL, "pkv_rope_create: inv_freq[%d] is not finite or above 2^20", i);
        if (pair_axis && (pair_axis[i] < 0 || pair_axis[i] >= n_axes))
            return fail(PKV_EINVAL, "pkv_rope_create: pair_axis[%d] = %d is not an axis (0..%d)", i, pair_axis[i],
                        n_axes - 1);
    }
    pkv_rope *r = new (std::nothrow) pkv_rope();
    if (!r) return fail(PKV_ENOMEM, "pkv_rope_create: host allocation failed");
    r->rot_dim = rot_dim;
    r->interleaved = interleaved;
    r->n_axes = n_axes;
    for (int i = 0; i < rot_dim / 2; ++i) {
        r->turn[i] = turn_fraction(inv_freq[i]);
        r->axis[i] = (uint8_t)(pair_axis ? pair_axis[i] : 0);
    }
    *out = r;
    return PKV_OK;
}

extern "C" pkv_status pkv_rope_destroy(pkv_rope *rope)
{
    delete rope;
    return PKV_OK;
}

extern "C" pkv_status paged_rope_append(pkv_pool *pool, const pkv_rope *rope, const void *q, int64_t q_stride,
                                        int32_t n_q, const void *k_new, int64_t k_stride, const void *v_new,
                                        int64_t v_stride, const int32_t *positions, const int64_t *slot_mapping,
                                        int64_t n_tokens, void *q_out, int64_t q_out_stride, void *stream)
{
    const char *who = "paged_rope_append";
    if (!pool) return fail(PKV_EINVAL, "%s: NULL pool", who);
    if (!rope) return fail(PKV_EINVAL, "%s: NULL rope", who);
    if (n_tokens < 0) return fail(PKV_EINVAL, "%s: n_tokens < 0", who);
    if (n_q < 0 || n_q > 4096) return fail(PKV_EINVAL, "%s: n_q %d not in 0..4096", who, n_q);
    if (rope->rot_dim > pool->d_head)
        return fail(PKV_EINVAL, "%s: rot_dim %d is above the pool's d_head %d", who, rope->rot_dim, pool->d_head);
    if (pool->dtype != PKV_BF16 && !pool->scales_set)
        return fail(PKV_EINVAL, "%s: quantised pool needs its scales first (kv_pool_set_fp8_scales or "
                    "kv_pool_set_int4_key_params)", who);
    if (n_tokens == 0) return PKV_OK;
    if (n_tokens > INT32_MAX) return fail(PKV_EUNSUPPORTED, "%s: more than 2^31 tokens", who);
    if (!k_new || !v_new || !positions || !slot_mapping || (n_q > 0 && (!q || !q_out)))
        return fail(PKV_EINVAL, "%s: NULL device pointer", who);
    const int64_t wq = (int64_t)n_q * pool->d_head, wkv = (int64_t)pool->n_kv * pool->d_head;
    if (k_stride < wkv || v_stride < wkv || (n_q > 0 && (q_stride < wq || q_out_stride < wq)))
        return fail(PKV_EINVAL, "%s: a token stride is smaller than the token's heads", who);
    const int64_t most = (int64_t)1 << 40;
    if (k_stride > most || v_stride > most || (n_q > 0 && (q_stride > most || q_out_stride > most)))
        return fail(PKV_EINVAL, "%s: a token stride is above 2^40 elements", who);
    if (((uintptr_t)k_new | (uintptr_t)v_new | (n_q > 0 ? (uintptr_t)q | (uintptr_t)q_out : 0)) & 15u)
        return fail(PKV_EINVAL, "%s: q, k_new, v_new and q_out must be 16-byte aligned", who);
    if ((k_stride | v_stride | (n_q > 0 ? q_stride | q_out_stride : 0)) & 7)
        return fail(PKV_EINVAL, "%s: token strides must be multiples of 8 elements", who);
    if (((uintptr_t)positions & 3u) || ((uintptr_t)slot_mapping & 7u))
        return fail(PKV_EINVAL, "%s: positions must be 4-byte and slot_mapping 8-byte aligned", who);
    if (n_q > 0) {  // other tokens' rows must not be overwritten before they are read
        if (!(q == q_out && q_stride == q_out_stride) &&
            rows_overlap(q, q_stride, wq, q_out, q_out_stride, wq, n_tokens))
            return fail(PKV_EINVAL, "%s: q_out overlaps q without being q itself", who);
        if (rows_overlap(k_new, k_stride, wkv, q_out, q_out_stride, wq, n_tokens) ||
            rows_overlap(v_new, v_stride, wkv, q_out, q_out_stride, wq, n_tokens))
            return fail(PKV_EINVAL, "%s: q_out overlaps k_new or v_new", who);
    }
    pkv_status st = check_pool_device(pool, who);
    if (st != PKV_OK) return st;

    RopeArgs a;
    for (int i = 0; i < 64; ++i) {
        a.turn[i] = rope->turn[i];
        a.axis[i] = rope->axis[i];
    }
    a.rot_dim = rope->rot_dim;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k_new);
    a.v = static_cast<const __nv_bfloat16 *>(v_new);
    a.q_out = static_cast<__nv_bfloat16 *>(q_out);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.qo_stride = q_out_stride;
    a.n_q = n_q;
    a.n_kv = pool->n_kv;
    a.positions = positions;
    a.slots = slot_mapping;
    a.n_tokens = n_tokens;
    a.pool = static_cast<uint8_t *>(pool->k);
    a.num_blocks = pool->num_blocks;
    a.scales = pool->scales;
    a.k_params = pool->k_params;
    a.err = pool->err;
    // Few tokens: a token's head rows are shared by several warps, one step of rows each at most,
    // until about 16 warps per SM run.
    const int rpw = 512 / pool->d_head;
    const int steps = (n_q + 2 * pool->n_kv + rpw - 1) / rpw;
    const int64_t want = ((int64_t)pool->num_sms * 16 + n_tokens - 1) / n_tokens;
    a.splits = (int)std::max<int64_t>(1, std::min<int64_t>(steps, want));
    const int64_t ctas = (n_tokens * a.splits + kRopeWarps - 1) / kRopeWarps;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LaunchScope ls(pool, kAppend, s);
    cudaError_t e = pool->d_head == 128 ? launch_kv<128>(a, pool->dtype, rope->interleaved != 0, ctas, s)
                                        : launch_kv<64>(a, pool->dtype, rope->interleaved != 0, ctas, s);
    ls.done();
    if (e != cudaSuccess) return cuda_fail(e, "paged_rope_append launch");
    return PKV_OK;
}
