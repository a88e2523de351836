// attn_paged.cu -- attention of each request's newest tokens over its paged cache.
//
// One warp per (token, query head): its lanes hold head_dim / 32 values each
// and walk the keys with the running maximum and sum of a softmax.
#include "kernels.h"
#include "kv.cuh"
#include "profile.h"

namespace dspark {

namespace {

constexpr int kWarps = 4;

struct PagedParams {
    const uint16_t* q;
    int64_t q_stride;
    const uint8_t* k;
    const uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    const int32_t* q_off;
    const int32_t* kv_len;
    const int32_t* page_table;
    uint16_t* out;
    float* lse;
    void* ws;
    int R, max_pages, T, n_pages, page_log2, heads, kv_heads;
    float scale2;                      // scale log2(e)
};

// N = head_dim / 32 values of a cached row
template <int N, bool F8>
__device__ __forceinline__ void load_row(const uint8_t* base, const float* scale, size_t row, int lane, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const size_t at = row * (N * 32) + lane * N + i;
        if (F8) {
            const uint2 b = e4m3x4_to_bf16x4(__ldg(base + at));
            x[i] = bf16_bits_to_float(b.x & 0xFFFFu) * __ldg(scale + row);
        } else {
            x[i] = bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t*>(base) + at));
        }
    }
}

template <int HD, bool F8>
__global__ void __launch_bounds__(kWarps * 32) attn_paged_kernel(PagedParams p) {
    constexpr int N = HD / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t most = (int64_t)p.max_pages << p.page_log2;
    if (blockIdx.x == 0) check_requests(p.q_off, p.kv_len, p.R, p.T, most, p.ws);
    const int t = (int)(w / p.heads), h = (int)(w % p.heads);
    if (t >= p.T) return;
    const int r = find_request(p.q_off, p.R, t);
    const RowRange rows = row_range(p.q_off, r, p.T);
    if (t < rows.a || t >= rows.b) return;
    const int seen = clamped_len(p.kv_len, r, most) - (rows.b - t) + 1;    // keys this token sees
    const int kvh = h / (p.heads / p.kv_heads);
    float q[N], o[N], k[N];
    const uint16_t* src = p.q + (size_t)t * p.q_stride + (size_t)h * HD + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        q[i] = bf16_bits_to_float(src[i]) * p.scale2;
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < seen; ++j) {
        const int page = __ldg(p.page_table + (size_t)r * p.max_pages + (j >> p.page_log2));
        const bool ok = page >= 0 && page < p.n_pages;
        if (!ok && lane == 0) raise_status(p.ws, kStatBadPage);
        const size_t row = (((size_t)(ok ? page : 0) * p.kv_heads + kvh) << p.page_log2) +
                           (j & ((1 << p.page_log2) - 1));
        float s = 0.f;
        if (ok) {
            load_row<N, F8>(p.k, p.k_scale, row, lane, k);
#pragma unroll
            for (int i = 0; i < N; ++i) s = fmaf(q[i], k[i], s);
        }
        s = warp_sum(s);
        const float mn = fmaxf(m, s), f = ex2_approx(m - mn), e = ex2_approx(s - mn);
        m = mn;
        l = fmaf(l, f, e);
        if (ok) load_row<N, F8>(p.v, p.v_scale, row, lane, k);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(o[i], f, ok ? e * k[i] : 0.f);
    }
    uint16_t* dst = p.out + ((size_t)t * p.heads + h) * HD + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) dst[i] = __bfloat16_as_ushort(__float2bfloat16_rn(seen > 0 ? o[i] / l : 0.f));
    if (p.lse && lane == 0)
        p.lse[(size_t)t * p.heads + h] = seen > 0 ? (float)((double)m * 0.6931471805599453 + log((double)l)) : -INFINITY;
}

}  // namespace

size_t attn_paged_workspace_bytes(int, int, int, int, int) { return sizeof(WsHeader); }

cudaError_t launch_attn_paged(const void* q, int64_t q_stride, const dspark_kv_cache_t& c, const dspark_kv_batch_t& b,
                              int n_heads, float scale, void* out, float* lse, void* ws, cudaStream_t s) {
    PagedParams p = {static_cast<const uint16_t*>(q), q_stride, static_cast<const uint8_t*>(c.k),
                     static_cast<const uint8_t*>(c.v), c.k_scale, c.v_scale, b.q_off, b.kv_len, b.page_table,
                     static_cast<uint16_t*>(out), lse, ws, b.R, b.max_pages, b.T, c.n_pages, ceil_log2_i(c.page),
                     n_heads, c.n_kv_heads, scale * kLog2e};
    const dim3 grid((unsigned)(((int64_t)b.T * n_heads + kWarps - 1) / kWarps)), block(kWarps * 32);
    const bool f8 = c.dtype == DSPARK_E4M3;
    auto kern = c.head_dim == 64 ? (f8 ? attn_paged_kernel<64, true> : attn_paged_kernel<64, false>)
                                 : (f8 ? attn_paged_kernel<128, true> : attn_paged_kernel<128, false>);
    prof_begin(kPAttnPaged, s);
    const cudaError_t e = launch_kernel(kern, grid, block, 0, s, false, p);
    prof_end(s);
    return e;
}

}  // namespace dspark
