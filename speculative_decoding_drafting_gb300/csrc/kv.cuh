// kv.cuh -- device helpers of the paged key-value cache: the requests of a
// call, their tokens' places, and e4m3 codes.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "sm100.cuh"

namespace dspark {

// Request r's rows [a, b) of a packed axis of T tokens; offsets outside
// [0, T] are clamped and decreasing ones make the request empty, so that
// every row index stays in range whatever the array holds.  (Plain loads: the
// read-only path may not see what a kernel wrote that this one overlaps.)
struct RowRange {
    int a, b;
};
__device__ __forceinline__ RowRange row_range(const int32_t* off, int r, int T) {
    const int a = min(max(off[r], 0), T), b = min(max(off[r + 1], 0), T);
    return RowRange{a, max(a, b)};
}
__device__ __forceinline__ int clamped_len(const int32_t* kv_len, int r, int64_t most) {
    return (int)min((int64_t)max(kv_len[r], 0), most);
}

// The last request whose offset is <= t (0 if none), by all 32 lanes of a
// warp: each round splits the range into 32 and takes two memory latencies
// for up to 1024 requests, against ten of a binary search.
__device__ __forceinline__ int find_request(const int32_t* off, int R, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = R;                           // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool le = at < lo + n && __ldg(off + at) <= t;
        const uint32_t m = __ballot_sync(0xffffffffu, le);
        const int k = m ? 31 - __clz(m) : 0;
        const int end = lo + n;
        lo += k * step;
        n = min(step, end - lo);
    }
    return lo;
}

// Records BAD_PAGE for offsets or lengths out of range (kv_len may be null);
// the threads of one CTA share the requests.
__device__ __forceinline__ void check_requests(const int32_t* off, const int32_t* kv_len, int R, int T, int64_t most,
                                               void* ws) {
    bool bad = false;
    for (int r = threadIdx.x; r < R; r += blockDim.x) {
        const int a = off[r], b = off[r + 1];
        bad |= a < 0 || b > T || b < a;
        if (kv_len) {
            const int n = kv_len[r];
            bad |= n < 0 || n > most;
        }
    }
    if (bad) raise_status(ws, kStatBadPage);
}

// e4m3 codes of two values y: bf16 values x times (448 / a) in float32 (packed
// pairs x, inv), the row's largest magnitude a (finite, above zero).  The code is the
// e4m3 value nearest to the exact quotient x 448 / a.  x and a have 8 significant
// bits and 448 = 7 2^6, so the quotient either lies on a midpoint of two e4m3
// values (5 significant bits) or at a relative distance above 2^-13 of it.
// t = x (448 / a) in float32 is within 2^-22 of the quotient; rounding t to 15
// significant bits (Veltkamp's splitting, T. J. Dekker, "A floating-point
// technique for extending the available precision", 1971) restores exact
// midpoints and moves no other value across one.
__device__ __forceinline__ uint32_t quantise2(uint64_t x, uint64_t inv) {
    const uint64_t k = pack2(513.f, 513.f), minus = pack2(-1.f, -1.f);
    const uint64_t t = mul2x(x, inv);
    const uint64_t c = mul2x(t, k);
    float2 y;
    unpack2(fma2(fma2(t, minus, c), minus, c), y.x, y.y);                 // c - (c - t)
    return __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
}
// The same of 8 bf16 values (w).
__device__ __forceinline__ uint2 quantise8(uint4 w, float inv) {
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    const uint64_t i2 = pack2(inv, inv);
    uint32_t half[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) half[i] = quantise2(pack2(bf16_bits_to_float(in[i] & 0xFFFFu), bf16_bits_to_float(in[i] >> 16)), i2);
    return make_uint2(half[0] | (half[1] << 16), half[2] | (half[3] << 16));
}

// bf16 bits of four e4m3 codes (bytes of w), exactly.  An e4m3 value with its
// sign, exponent and fraction bits moved to bf16's places is the value times
// 2^-120 (the exponent biases are 7 and 127; an e4m3 subnormal becomes a bf16
// subnormal), so one exact bf16 product by 2^120 finishes it.  The NaN codes
// 0x7F and 0xFF, which the cache writer never stores, read as +-480.
__device__ __forceinline__ uint2 e4m3x4_to_bf16x4(uint32_t w) {
    // bytes 0, 1 -> lo; 2, 3 -> hi, each byte in the upper half of a 16-bit lane
    const uint32_t lo = __byte_perm(w, 0u, 0x1404), hi = __byte_perm(w, 0u, 0x3424);
    const uint32_t a = (lo & 0x80008000u) | ((lo & 0x7F007F00u) >> 4);
    const uint32_t b = (hi & 0x80008000u) | ((hi & 0x7F007F00u) >> 4);
    const __nv_bfloat162 k = __floats2bfloat162_rn(1.329227995784916e36f, 1.329227995784916e36f);   // 2^120
    const __nv_bfloat162 ra = __hmul2(reinterpret_cast<const __nv_bfloat162&>(a), k);
    const __nv_bfloat162 rb = __hmul2(reinterpret_cast<const __nv_bfloat162&>(b), k);
    return make_uint2(reinterpret_cast<const uint32_t&>(ra), reinterpret_cast<const uint32_t&>(rb));
}

// Eight e4m3 codes (bytes of a, then of b) as fp16, exactly.
__device__ __forceinline__ uint4 e4m3x8_to_half8(uint32_t a, uint32_t b) {
    auto two = [](uint32_t w) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3);
        return (uint32_t)h.x | ((uint32_t)h.y << 16);
    };
    return make_uint4(two(a & 0xFFFFu), two(a >> 16), two(b & 0xFFFFu), two(b >> 16));
}

}  // namespace dspark
