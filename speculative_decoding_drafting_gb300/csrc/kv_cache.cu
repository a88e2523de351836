// kv_cache.cu -- writing new tokens' keys and values into the paged cache
// (bf16, or e4m3 with a float32 scale per token and head) and reading them back.
//
// Both move each row once and are bound by its bytes: a row is head_dim values
// of one token and head, 8 or 16 lanes hold 8 values each (16 bytes of bf16),
// and a warp takes one token with all its heads, K and V, so that its loads
// are in flight together.  Measured (GB300, against 6.68 TB/s of a plain copy;
// 8 heads of 128): 47386 tokens into an e4m3 cache 52.4 us, 5.6 TB/s; 109747
// tokens out of one 104.6 us, 6.5 TB/s.  (With K's rows used up before V's were
// loaded and a division per lane it was 69.8 and 127 us.)
#include <type_traits>

#include "kernels.h"
#include "kv.cuh"
#include "profile.h"
#include "sm100.cuh"

namespace dspark {

namespace {

constexpr int kWarps = 4;          // tokens per CTA

__device__ __forceinline__ uint32_t bf16x2_abs_bits(uint32_t w) { return w & 0x7FFF7FFFu; }

// Codes of 8 bf16 values (w) with the row's largest magnitude a (float bits
// of a finite value > 0).  The code is the e4m3 value nearest to the exact
// quotient x 448 / a.  x and a have 8 significant bits and 448 = 7 2^6, so the
// quotient either lies on a midpoint of two e4m3 values (5 significant bits)
// or at a relative distance above 2^-13 of it.  t = x (448 / a) in float32 is
// within 2^-22 of the quotient; rounding t to 15 significant bits (Veltkamp's
// splitting, T. J. Dekker, "A floating-point technique for extending the
// available precision", 1971) restores exact midpoints and moves no other
// value across one.
__device__ __forceinline__ uint2 quantise8(uint4 w, float inv) {
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    const uint64_t k = pack2(513.f, 513.f), i2 = pack2(inv, inv), minus = pack2(-1.f, -1.f);
    uint32_t half[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t t = mul2x(pack2(bf16_bits_to_float(in[i] & 0xFFFFu), bf16_bits_to_float(in[i] >> 16)), i2);
        const uint64_t c = mul2x(t, k);
        float2 y;
        unpack2(fma2(fma2(t, minus, c), minus, c), y.x, y.y);             // c - (c - t)
        half[i] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(half[0] | (half[1] << 16), half[2] | (half[3] << 16));
}

// A warp's row vectors of one step: kSteps of K, then kSteps of V.
constexpr int kSteps = 4, kVecs = 2 * kSteps;

// The largest of each of the kVecs values over the LANES lanes of a row: lane
// `part` gets the one of vector part / (LANES / kVecs).  Each exchange halves
// the vectors, 7 or 8 exchanges where one reduction per vector takes 24 or 32.
template <int LANES>
__device__ __forceinline__ uint32_t row_maxima(uint32_t (&m)[kVecs], int part) {
#pragma unroll
    for (int n = kVecs / 2, o = LANES / 2; n > 0; n >>= 1, o >>= 1) {
        const bool upper = part & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint32_t give = upper ? m[i] : m[i + n], keep = upper ? m[i + n] : m[i];
            m[i] = __vmaxu2(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
    }
#pragma unroll
    for (int o = LANES / 16; o > 0; o >>= 1) m[0] = __vmaxu2(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
    return m[0];
}

struct WriteParams {
    const uint16_t* src[2];        // K, V
    int64_t stride[2];
    uint8_t* dst[2];
    float* scale[2];
    const int32_t* q_off;
    const int32_t* kv_len;
    const int32_t* page_table;
    void* ws;
    int R, max_pages, T, n_pages, page_log2, heads;
};

template <int HD, bool F8>
__global__ void __launch_bounds__(kWarps * 32) kv_write_kernel(WriteParams p) {
    constexpr int kLanes = HD / 8;                  // lanes of a row
    constexpr int kRows = 32 / kLanes;              // heads per warp instruction
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t most = (int64_t)p.max_pages << p.page_log2;
    if (blockIdx.x == gridDim.x - 1) check_requests(p.q_off, p.kv_len, p.R, p.T, most, p.ws);
    if (t >= p.T) return;
    const int sub = lane / kLanes, part = lane % kLanes;
    const int r = find_request(p.q_off, p.R, t);
    const RowRange rows = row_range(p.q_off, r, p.T);
    const int pos = clamped_len(p.kv_len, r, most) - (rows.b - t);
    if (t < rows.a || t >= rows.b || pos < 0) return;
    const int page = __ldg(p.page_table + (size_t)r * p.max_pages + (pos >> p.page_log2));
    if (page < 0 || page >= p.n_pages) {
        if (lane == 0) raise_status(p.ws, kStatBadPage);
        return;
    }
    const int slot = pos & ((1 << p.page_log2) - 1);
    const size_t row0 = (((size_t)page * p.heads) << p.page_log2) + slot;    // head 0's row of the cache
    for (int h0 = 0; h0 < p.heads; h0 += kSteps * kRows) {
        // K's and V's loads are all in flight before the first is used
        uint4 w[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int kv = i / kSteps, h = h0 + (i % kSteps) * kRows + sub;
            w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (h < p.heads)
                w[i] = __ldcs(reinterpret_cast<const uint4*>(p.src[kv] + (size_t)t * p.stride[kv] + (size_t)h * HD + part * 8));
        }
        float inv = 0.f;
        if (F8) {
            // largest magnitude of a row: bf16 magnitudes order as their bits do
            // (a NaN's lie above infinity's)
            uint32_t m[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                m[i] = __vmaxu2(__vmaxu2(bf16x2_abs_bits(w[i].x), bf16x2_abs_bits(w[i].y)),
                                __vmaxu2(bf16x2_abs_bits(w[i].z), bf16x2_abs_bits(w[i].w)));
            // each lane now takes one row: one scale and one reciprocal for all the
            // warp's rows, where every lane would divide for its own vectors
            const uint32_t big = row_maxima<kLanes>(m, part);
            const float a = bf16_bits_to_float(max(big & 0xFFFFu, big >> 16));
            const int i = part / (kLanes / kVecs), kv = i / kSteps, h = h0 + (i % kSteps) * kRows + sub;
            if (part % (kLanes / kVecs) == 0 && h < p.heads) p.scale[kv][row0 + ((size_t)h << p.page_log2)] = __fdiv_rn(a, 448.f);
            // below 2^-100 the reciprocal would overflow float32: such rows (a
            // negative sign marks them) are scaled up by 2^64 first, which changes
            // no quotient; rows that are zero or not finite get codes of zero
            if (a > 0.f && a < INFINITY)
                inv = a < 7.888609e-31f ? -__fdiv_rn(448.f, a * 1.8446744e19f) : __fdiv_rn(448.f, a);
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int kv = i / kSteps, h = h0 + (i % kSteps) * kRows + sub;
            const size_t row = row0 + ((size_t)h << p.page_log2);
            if (!F8) {
                if (h < p.heads) *reinterpret_cast<uint4*>(p.dst[kv] + (row * HD + part * 8) * 2) = w[i];
                continue;
            }
            const float f = __shfl_sync(0xffffffffu, inv, sub * kLanes + i * (kLanes / kVecs));
            if (f < 0.f) {
                uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                const __nv_bfloat162 up = __floats2bfloat162_rn(1.8446744e19f, 1.8446744e19f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 y = __hmul2(reinterpret_cast<const __nv_bfloat162&>(x[e]), up);
                    x[e] = reinterpret_cast<const uint32_t&>(y);
                }
                w[i] = make_uint4(x[0], x[1], x[2], x[3]);
            }
            uint2 code = quantise8(w[i], fabsf(f));
            if (f == 0.f) code = make_uint2(0u, 0u);
            if (h < p.heads) *reinterpret_cast<uint2*>(p.dst[kv] + row * HD + part * 8) = code;
        }
    }
}

struct ReadParams {
    const uint8_t* src[2];
    const float* scale[2];
    uint16_t* dst[2];
    const int32_t* off;
    const int32_t* page_table;
    void* ws;
    int R, max_pages, T, n_pages, page_log2, heads;
};

template <int HD, bool F8>
__global__ void __launch_bounds__(kWarps * 32) kv_read_kernel(ReadParams p) {
    constexpr int kLanes = HD / 8;
    constexpr int kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t most = (int64_t)p.max_pages << p.page_log2;
    if (blockIdx.x == gridDim.x - 1) {
        check_requests(p.off, nullptr, p.R, p.T, most, p.ws);
        for (int r = threadIdx.x; r < p.R; r += blockDim.x) {
            const RowRange rows = row_range(p.off, r, p.T);
            if (rows.b - rows.a > most) raise_status(p.ws, kStatBadPage);
        }
    }
    if (t >= p.T) return;
    const int sub = lane / kLanes, part = lane % kLanes;
    const int r = find_request(p.off, p.R, t);
    const RowRange rows = row_range(p.off, r, p.T);
    const int pos = t - rows.a;
    if (pos < 0 || t >= rows.b) return;
    const int page = pos < most ? __ldg(p.page_table + (size_t)r * p.max_pages + (pos >> p.page_log2)) : -1;
    const bool ok = page >= 0 && page < p.n_pages;
    if (!ok && lane == 0) raise_status(p.ws, kStatBadPage);
    const int slot = pos & ((1 << p.page_log2) - 1);
    const size_t row0 = (((size_t)(ok ? page : 0) * p.heads) << p.page_log2) + slot;
    for (int h0 = 0; h0 < p.heads; h0 += kSteps * kRows) {
        // K's and V's loads are all in flight before the first is used
        using Vec = std::conditional_t<F8, uint2, uint4>;
        Vec w[kVecs];
        float scale[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int kv = i / kSteps, h = h0 + (i % kSteps) * kRows + sub;
            const size_t row = row0 + ((size_t)h << p.page_log2);
            w[i] = Vec{};
            scale[i] = 0.f;
            if (!ok || h >= p.heads) continue;
            w[i] = __ldcs(reinterpret_cast<const Vec*>(p.src[kv] + row * HD * (F8 ? 1 : 2) + part * sizeof(Vec)));
            if (F8) scale[i] = __ldg(p.scale[kv] + row);
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int kv = i / kSteps, h = h0 + (i % kSteps) * kRows + sub;
            if (h >= p.heads) continue;
            uint4 o;
            if constexpr (F8) {
                const uint2 a = e4m3x4_to_bf16x4(w[i].x), b = e4m3x4_to_bf16x4(w[i].y);
                const uint32_t x[4] = {a.x, a.y, b.x, b.y};
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(bf16_bits_to_float(x[e] & 0xFFFFu) * scale[i],
                                                                   bf16_bits_to_float(x[e] >> 16) * scale[i]);
                    y[e] = reinterpret_cast<const uint32_t&>(v);
                }
                o = make_uint4(y[0], y[1], y[2], y[3]);
            } else {
                o = w[i];
            }
            __stcs(reinterpret_cast<uint4*>(p.dst[kv] + ((size_t)t * p.heads + h) * HD + part * 8), o);
        }
    }
}

int log2_of(int x) { return ceil_log2_i(x); }

}  // namespace

cudaError_t launch_kv_write(const dspark_kv_cache_t& c, const dspark_kv_batch_t& b, const void* K, const void* V,
                            int64_t k_stride, int64_t v_stride, void* ws, cudaStream_t s) {
    WriteParams p = {{static_cast<const uint16_t*>(K), static_cast<const uint16_t*>(V)},
                     {k_stride, v_stride},
                     {static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v)},
                     {c.k_scale, c.v_scale},
                     b.q_off, b.kv_len, b.page_table, ws,
                     b.R, b.max_pages, b.T, c.n_pages, log2_of(c.page), c.n_kv_heads};
    const dim3 grid((unsigned)((b.T + kWarps - 1) / kWarps)), block(kWarps * 32);
    const bool f8 = c.dtype == DSPARK_E4M3;
    auto kern = c.head_dim == 64 ? (f8 ? kv_write_kernel<64, true> : kv_write_kernel<64, false>)
                                 : (f8 ? kv_write_kernel<128, true> : kv_write_kernel<128, false>);
    prof_begin(kPKvWrite, s);
    const cudaError_t e = launch_kernel(kern, grid, block, 0, s, false, p);
    prof_end(s);
    return e;
}

cudaError_t launch_kv_read(const dspark_kv_cache_t& c, const dspark_kv_batch_t& b, void* K, void* V, void* ws,
                           cudaStream_t s) {
    ReadParams p = {{static_cast<const uint8_t*>(c.k), static_cast<const uint8_t*>(c.v)},
                    {c.k_scale, c.v_scale},
                    {static_cast<uint16_t*>(K), static_cast<uint16_t*>(V)},
                    b.q_off, b.page_table, ws,
                    b.R, b.max_pages, b.T, c.n_pages, log2_of(c.page), c.n_kv_heads};
    const dim3 grid((unsigned)((b.T + kWarps - 1) / kWarps)), block(kWarps * 32);
    const bool f8 = c.dtype == DSPARK_E4M3;
    auto kern = c.head_dim == 64 ? (f8 ? kv_read_kernel<64, true> : kv_read_kernel<64, false>)
                                 : (f8 ? kv_read_kernel<128, true> : kv_read_kernel<128, false>);
    prof_begin(kPKvRead, s);
    const cudaError_t e = launch_kernel(kern, grid, block, 0, s, false, p);
    prof_end(s);
    return e;
}

}  // namespace dspark
