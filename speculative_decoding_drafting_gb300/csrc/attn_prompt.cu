// attn_prompt.cu -- causal attention over whole prompts, packed one after another.
//
// One warp per (token, query head): its lanes hold head_dim / 32 values each
// and walk the keys with the running maximum and sum of a softmax.
#include "kernels.h"
#include "kv.cuh"
#include "profile.h"

namespace dspark {

namespace {

constexpr int kWarps = 4;

template <int HD>
__global__ void __launch_bounds__(kWarps * 32) attn_prompt_kernel(PromptArgs p) {
    constexpr int N = HD / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (blockIdx.x == 0) check_requests(p.seq_off, nullptr, p.B, p.T, 0, p.ws);
    const int t = (int)(w / p.n_heads), h = (int)(w % p.n_heads);
    if (t >= p.T) return;
    const int b = find_request(p.seq_off, p.B, t);
    const RowRange rows = row_range(p.seq_off, b, p.T);
    if (t < rows.a || t >= rows.b) return;
    const int kvh = h / (p.n_heads / p.n_kv_heads);
    const float scale2 = p.scale * kLog2e;
    float q[N], o[N];
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + (size_t)t * p.q_stride + (size_t)h * HD + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        q[i] = bf16_bits_to_float(src[i]) * scale2;
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const uint16_t* k = static_cast<const uint16_t*>(p.k) + (size_t)kvh * HD + lane * N;
    const uint16_t* v = static_cast<const uint16_t*>(p.v) + (size_t)kvh * HD + lane * N;
    for (int j = rows.a; j <= t; ++j) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) s = fmaf(q[i], bf16_bits_to_float(__ldg(k + (size_t)j * p.k_stride + i)), s);
        s = warp_sum(s);
        const float mn = fmaxf(m, s), f = ex2_approx(m - mn), e = ex2_approx(s - mn);
        m = mn;
        l = fmaf(l, f, e);
#pragma unroll
        for (int i = 0; i < N; ++i)
            o[i] = fmaf(o[i], f, e * bf16_bits_to_float(__ldg(v + (size_t)j * p.v_stride + i)));
    }
    uint16_t* dst = static_cast<uint16_t*>(p.out) + ((size_t)t * p.n_heads + h) * HD + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) dst[i] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i] / l));
    if (p.lse && lane == 0) p.lse[(size_t)t * p.n_heads + h] = (float)((double)m * 0.6931471805599453 + log((double)l));
}

}  // namespace

size_t attn_prompt_workspace_bytes(int, int, int, int, int) { return sizeof(WsHeader); }

cudaError_t launch_attn_prompt(const PromptArgs& a, cudaStream_t s) {
    const dim3 grid((unsigned)(((int64_t)a.T * a.n_heads + kWarps - 1) / kWarps)), block(kWarps * 32);
    auto kern = a.head_dim == 64 ? attn_prompt_kernel<64> : attn_prompt_kernel<128>;
    prof_begin(kPAttnPrompt, s);
    const cudaError_t e = launch_kernel(kern, grid, block, 0, s, false, a);
    prof_end(s);
    return e;
}

}  // namespace dspark
