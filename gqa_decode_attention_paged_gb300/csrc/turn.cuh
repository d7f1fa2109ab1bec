// Angles as fractions of a turn.  Plain C++ as well as CUDA, so that it can be
// checked without a GPU.
#pragma once

#include <math.h>
#include <stdint.h>

#ifdef __CUDACC__
#define PKV_ANGLE_FN __host__ __device__ __forceinline__
#else
#define PKV_ANGLE_FN inline
#endif

namespace pkv {

// frac(f / 2 pi) 2^64, rounded to nearest, for |f| <= 2^20 (radians per position): f's 53 bits times the first 128
// bits of 1 / 2 pi.  What those leave off is below 2^-75 of a turn, and the rounding is 2^-65: at 2^31 positions
// 2^-34.  (The product in double is off by up to 2^-56 at f = 1, which is 2^-25 there.)
inline uint64_t turn_fraction(double f)
{
    constexpr uint64_t kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;  // 2^128 / 2 pi
    int e;
    const uint64_t m = (uint64_t)ldexp(frexp(fabs(f), &e), 53);  // |f| = m 2^(e - 53)
    const unsigned __int128 low = (unsigned __int128)m * kLow, high = (unsigned __int128)m * kHigh + (uint64_t)(low >> 64);
    const uint64_t w[4] = {(uint64_t)low, (uint64_t)high, (uint64_t)(high >> 64), 0};  // m 2^128 / 2 pi
    // the fraction's 64 bits are those from 2^(117 - e) on (e <= 21), and the one below rounds them
    const int at = 116 - e;
    if (at >= 192) return 0;
    const int i = at / 64, s = at % 64;
    const uint64_t next = i + 1 < 4 ? w[i + 1] : 0, after = i + 2 < 4 ? w[i + 2] : 0;
    const uint64_t below = s ? (w[i] >> s) | (next << (64 - s)) : w[i];  // 64 bits from `at`
    const uint64_t top = s ? (next >> s) | (after << (64 - s)) : next;   // and the 64 behind them
    const uint64_t turn = ((below >> 1) | (top << 63)) + (below & 1u);
    return f < 0.0 ? 0 - turn : turn;
}

// Sine and cosine of u 2^-32 turns: the nearest quarter turn is taken off as an integer, and the rest t, within
// pi / 4, goes into the Taylor series of both, with what its 24 bits cannot hold (lo) and with the rounding of the
// cosine's second sum.  Off by 0.726 of a last place at most, 0.251 in the mean, over all 2^32 angles, on the GPU and
// on the host (rounding alone: 0.5 and 0.25); as fast as sincospif of the rounded angle, which is off by up to 2.
PKV_ANGLE_FN void turn_of(uint32_t u, float &sn, float &cs)
{
    constexpr float kPi = 3.14159274f, kPiRest = -8.74227766e-8f;  // pi and what its rounding leaves
    const uint32_t quarter = (u + 0x20000000u) >> 30;
    const int32_t rest = (int32_t)(u - (quarter << 30));  // within 2^29
    const float n = (float)rest;
    const float x = n * 4.656612873077393e-10f;  // 2^-31 half turns
    const float t = x * kPi;
    const float lo = fmaf(x, kPi, -t) + fmaf(x, kPiRest, (float)(rest - (int32_t)n) * (kPi * 4.656612873077393e-10f));
    const float z = t * t, zl = fmaf(t, t, -z);
    float p = fmaf(z, 1.0f / 362880, -1.0f / 5040);
    p = fmaf(p, z, 1.0f / 120);
    p = fmaf(p, z, -1.0f / 6);
    const float s = t + fmaf(t * z, p, fmaf(-0.5f * z, lo, lo));
    float q = fmaf(z, -1.0f / 3628800, 1.0f / 40320);
    q = fmaf(q, z, -1.0f / 720);
    q = fmaf(q, z, 1.0f / 24);
    const float w = 1.0f - 0.5f * z, e = (1.0f - w) - 0.5f * z;  // (exact)
    const float c = w + (e + fmaf(z * z, q, fmaf(-lo, t, -0.5f * zl)));
    const float a = quarter & 1u ? c : s, b = quarter & 1u ? s : c;
    sn = quarter & 2u ? -a : a;
    cs = (quarter + 1u) & 2u ? -b : b;
}

}  // namespace pkv
