// kv_cache.cu -- writing new tokens' keys and values into the paged cache
// (bf16, or e4m3 with a float32 scale per token and head) and reading them back.
//
// Both move each row once: a row is head_dim values of one token and head, 8
// or 16 lanes hold 8 values each (16 bytes of bf16), and a warp takes one
// token with all its heads, K and V, so that its loads are in flight together.
#include "kernels.h"
#include "kv.cuh"
#include "profile.h"

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
    uint32_t out[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t half[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t x = in[2 * h + i];
            float2 t = make_float2(bf16_bits_to_float(x & 0xFFFFu) * inv, bf16_bits_to_float(x >> 16) * inv);
            const float cx = t.x * 513.f, cy = t.y * 513.f;
            t.x = __fsub_rn(cx, __fsub_rn(cx, t.x));
            t.y = __fsub_rn(cy, __fsub_rn(cy, t.y));
            half[i] = __nv_cvt_float2_to_fp8x2(t, __NV_SATFINITE, __NV_E4M3);
        }
        out[h] = half[0] | (half[1] << 16);
    }
    return make_uint2(out[0], out[1]);
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
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const uint16_t* src = p.src[kv] + (size_t)t * p.stride[kv];
#pragma unroll 4
        for (int h0 = 0; h0 < p.heads; h0 += kRows) {
            const int h = h0 + sub;
            const bool in = h < p.heads;
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (in) w = __ldcs(reinterpret_cast<const uint4*>(src + (size_t)h * HD + part * 8));
            const size_t row = row0 + ((size_t)h << p.page_log2);
            if (!F8) {
                if (in) *reinterpret_cast<uint4*>(p.dst[kv] + (row * HD + part * 8) * 2) = w;
                continue;
            }
            // largest magnitude of the row: bf16 magnitudes order as their bits do
            // (a NaN's lie above infinity's)
            uint32_t m = __vmaxu2(__vmaxu2(bf16x2_abs_bits(w.x), bf16x2_abs_bits(w.y)),
                                  __vmaxu2(bf16x2_abs_bits(w.z), bf16x2_abs_bits(w.w)));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float a = bf16_bits_to_float(max(m & 0xFFFFu, m >> 16));
            const float scale = __fdiv_rn(a, 448.f);
            uint2 code = make_uint2(0u, 0u);
            // below 2^-100 the reciprocal would overflow float32: such rows are
            // scaled up by 2^64 first, which changes no quotient
            const bool tiny = a < 7.888609e-31f;
            if (a > 0.f && a < INFINITY) {
                if (!tiny) {
                    code = quantise8(w, __fdiv_rn(448.f, a));
                } else {
                    uint32_t x[4] = {w.x, w.y, w.z, w.w};
                    const __nv_bfloat162 up = __floats2bfloat162_rn(1.8446744e19f, 1.8446744e19f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 y = __hmul2(reinterpret_cast<const __nv_bfloat162&>(x[i]), up);
                        x[i] = reinterpret_cast<const uint32_t&>(y);
                    }
                    code = quantise8(make_uint4(x[0], x[1], x[2], x[3]), __fdiv_rn(448.f, a * 1.8446744e19f));
                }
            }
            if (in) {
                *reinterpret_cast<uint2*>(p.dst[kv] + row * HD + part * 8) = code;
                if (part == 0) p.scale[kv][row] = scale;
            }
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
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        uint16_t* dst = p.dst[kv] + (size_t)t * p.heads * HD;
#pragma unroll 4
        for (int h0 = 0; h0 < p.heads; h0 += kRows) {
            const int h = h0 + sub;
            if (h >= p.heads) continue;
            const size_t row = row0 + ((size_t)h << p.page_log2);
            uint4 o = make_uint4(0u, 0u, 0u, 0u);
            if (ok && !F8) o = __ldcs(reinterpret_cast<const uint4*>(p.src[kv] + (row * HD + part * 8) * 2));
            if (ok && F8) {
                const uint2 c = __ldcs(reinterpret_cast<const uint2*>(p.src[kv] + row * HD + part * 8));
                const float s = __ldg(p.scale[kv] + row);
                const uint2 a = e4m3x4_to_bf16x4(c.x), b = e4m3x4_to_bf16x4(c.y);
                const uint32_t x[4] = {a.x, a.y, b.x, b.y};
                uint32_t y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(bf16_bits_to_float(x[i] & 0xFFFFu) * s,
                                                                   bf16_bits_to_float(x[i] >> 16) * s);
                    y[i] = reinterpret_cast<const uint32_t&>(v);
                }
                o = make_uint4(y[0], y[1], y[2], y[3]);
            }
            __stcs(reinterpret_cast<uint4*>(dst + (size_t)h * HD + part * 8), o);
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
