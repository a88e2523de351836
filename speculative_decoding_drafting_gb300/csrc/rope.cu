// rope.cu -- query and key heads normed and turned to their positions, packed
// rows in and out, or keys and values on into the paged cache.
//
// A head x of head_dim values becomes y = x w / sqrt(mean x^2 + eps) (where there
// is a norm), and its first `rot` values are turned in pairs (a, b):
//   a' = a cos t - b sin t,  b' = b cos t + a sin t,  t = position x inv_freq
// The turns of a position are the fraction of position x (inv_freq / 2 pi), which
// a 64-bit integer product of the position and the frequency in units of 2^-64
// turns gives exactly, however far the position; cosine and sine of it are
// float32, and everything up to the one rounding of a stored value is float32.
//
// Bound by the bytes: each value is read and written once.  Lanes hold 8 values
// of a head, 4 and the 4 that they are turned with, so that neither a shuffle
// nor a second load is needed; 16 lanes share a head of 128 (8 one of 64).  A
// warp takes a token, works out its angles once (each lane 4 / (32 / lanes of a
// head) of the 4 that it needs) and goes through the token's heads, 8 vectors of
// 32 lanes at a time, all of their loads in flight before the first is used.
// With few tokens several warps share one.
#include <algorithm>
#include <cmath>

#include "kernels.h"
#include "kv.cuh"
#include "profile.h"
#include "sm100.cuh"

namespace dspark {

namespace {

constexpr int kWarps = 4;
constexpr int kVecs = 8;               // vectors of a chunk: 8 of q's or k's heads, or 4 of k's and 4 of v's
constexpr float kTiny = 0x1p-100f;

enum Mode : int { kRows = 0, kAppendBf16 = 1, kAppendE4m3 = 2 };

struct RopeParams {
    const uint16_t* src[3];            // q, k, v
    int64_t src_stride[3];
    uint16_t* out[2];                  // q, k as rows (k: null if not asked for)
    int64_t out_stride[2];
    int heads[2];                      // of q, of k and v
    const void* w[2];                  // norm weights of q, of k (null: no norm)
    int w_dtype;
    float eps;
    const int32_t* positions;          // null: the token's place in its request
    int n_axes, rot;
    float amplitude;
    int T, parts;                      // warps of a token
    // the cache
    uint8_t* dst[2];
    float* scale[2];
    const int32_t *q_off, *kv_len, *page_table;
    void* ws;
    int R, max_pages, n_pages, page_log2;
    uint64_t turn[64];                 // turns per position, in 2^-64
    uint8_t axis[64];
};

// N values per lane, each of another row of the LANES lanes: lane `part` gets the
// result of vector part / (LANES / N).  Each exchange halves the vectors.  (A row
// is joined in the same order whichever vector it is, and for any N.)
template <int N, int LANES, typename Op>
__device__ __forceinline__ float join_rows(float (&m)[N], int part, Op op) {
#pragma unroll
    for (int n = N / 2, o = LANES / 2; n > 0; n >>= 1, o >>= 1) {
        const bool upper = part & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = upper ? m[i] : m[i + n], keep = upper ? m[i + n] : m[i];
            m[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
    }
#pragma unroll
    for (int o = LANES / (2 * N); o > 0; o >>= 1) m[0] = op(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
    return m[0];
}

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t two_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return reinterpret_cast<const uint32_t&>(h);
}

// A lane's place in a head: values o0 .. o0 + 3 and o1 .. o1 + 3.  Value e of the
// first four is turned with value e of the second, or, in neighbouring pairs
// (kPairs: o1 = o0 + 4), even values with the odd ones after them.
template <int HD, bool kPairs>
struct Place {
    static constexpr int kLanes = HD / 8;
    static constexpr int kHeads = 32 / kLanes;                // heads of a vector
    int part, sub, o0, o1;
    bool turns;
    float c[4], s[4];

    __device__ __forceinline__ Place(int lane, int rot) : part(lane % kLanes), sub(lane / kLanes) {
        const int n = rot / 8;                                // lanes that turn
        turns = part < n;
        if (kPairs) {
            o0 = 8 * part;
            o1 = o0 + 4;
        } else {
            o0 = turns ? 4 * part : rot + 8 * (part - n);
            o1 = turns ? rot / 2 + 4 * part : o0 + 4;
        }
    }
    __device__ __forceinline__ void load(const uint16_t* row, uint32_t (&w)[4]) const {
        if (kPairs) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4*>(row + o0));
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const uint2 a = __ldcs(reinterpret_cast<const uint2*>(row + o0)), b = __ldcs(reinterpret_cast<const uint2*>(row + o1));
            w[0] = a.x, w[1] = a.y, w[2] = b.x, w[3] = b.y;
        }
    }
    // the first and second values of the four pairs
    __device__ __forceinline__ static void split(const uint32_t (&w)[4], float (&a)[4], float (&b)[4]) {
        if (kPairs) {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = lo16(w[e]), b[e] = hi16(w[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                a[2 * e] = lo16(w[e]), a[2 * e + 1] = hi16(w[e]);
                b[2 * e] = lo16(w[2 + e]), b[2 * e + 1] = hi16(w[2 + e]);
            }
        }
    }
    // a head's values times r and the weights (first and second of the pairs), turned
    __device__ __forceinline__ void turn(const uint32_t (&w)[4], bool norm, float r, const float (&wa)[4], const float (&wb)[4],
                                         float (&a)[4], float (&b)[4]) const {
        split(w, a, b);
        if (norm) {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] *= r * wa[e], b[e] *= r * wb[e];
        }
        if (turns) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = a[e], y = b[e];
                a[e] = fmaf(x, c[e], -(y * s[e]));
                b[e] = fmaf(y, c[e], x * s[e]);
            }
        }
    }
    __device__ __forceinline__ void store(uint16_t* row, const float (&a)[4], const float (&b)[4]) const {
        if (kPairs)
            *reinterpret_cast<uint4*>(row + o0) =
                make_uint4(two_bf16(a[0], b[0]), two_bf16(a[1], b[1]), two_bf16(a[2], b[2]), two_bf16(a[3], b[3]));
        else {
            *reinterpret_cast<uint2*>(row + o0) = make_uint2(two_bf16(a[0], a[1]), two_bf16(a[2], a[3]));
            *reinterpret_cast<uint2*>(row + o1) = make_uint2(two_bf16(b[0], b[1]), two_bf16(b[2], b[3]));
        }
    }
    __device__ __forceinline__ void weights(const void* w, int dtype, float (&a)[4], float (&b)[4]) const {
        if (dtype == DSPARK_F32) {
            const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + o0));
            const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + o1));
            if (kPairs)
                a[0] = u.x, b[0] = u.y, a[1] = u.z, b[1] = u.w, a[2] = v.x, b[2] = v.y, a[3] = v.z, b[3] = v.w;
            else
                a[0] = u.x, a[1] = u.y, a[2] = u.z, a[3] = u.w, b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
        } else {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + o0));
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + o1));
            const uint32_t x[4] = {u.x, u.y, v.x, v.y};
            split(x, a, b);
        }
    }
};

template <int HD, bool kPairs, int MODE>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const __grid_constant__ RopeParams p) {
    using P = Place<HD, kPairs>;
    constexpr int kLanes = P::kLanes, kHeads = P::kHeads;
    constexpr int kOwn = 4 / kHeads;                          // angles that a lane works out
    const int lane = threadIdx.x & 31;
    P at(lane, p.rot);
    const int64_t most = (int64_t)p.max_pages << p.page_log2;
    if (MODE != kRows && blockIdx.x == gridDim.x - 1) check_requests(p.q_off, p.kv_len, p.R, p.T, most, p.ws);

    uint64_t turn[kOwn];
    int axis[kOwn];
#pragma unroll
    for (int e = 0; e < kOwn; ++e) {
        const int f = at.part * 4 + at.sub * kOwn + e;
        turn[e] = p.turn[f];
        axis[e] = p.axis[f];
    }
    const int q_chunks = (p.heads[0] + kVecs * kHeads - 1) / (kVecs * kHeads);
    const int kv_step = (MODE == kRows ? kVecs : kVecs / 2) * kHeads;
    const int chunks = q_chunks + (p.heads[1] + kv_step - 1) / kv_step;

    const int64_t warps = (int64_t)gridDim.x * kWarps;
    for (int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); task < (int64_t)p.T * p.parts; task += warps) {
        const int t = p.parts == 1 ? (int)task : (int)((uint32_t)task / (uint32_t)p.parts);
        bool known = false, in = true;
        int64_t slot_row = -1;                                // row of head 0 in the cache (in units of heads' rows)
        // the token's request, place and angles, while the first chunk's loads are in flight
        auto look = [&]() {
            known = true;
            int pos = 0;
            if (MODE != kRows) {
                const int r = find_request(p.q_off, p.R, t);
                const RowRange rows = row_range(p.q_off, r, p.T);
                in = t >= rows.a && t < rows.b;
                if (!in) return;
                pos = clamped_len(p.kv_len, r, most) - (rows.b - t);
                if (pos >= 0 && p.heads[1] > 0) {
                    const int page = __ldg(p.page_table + (size_t)r * p.max_pages + (pos >> p.page_log2));
                    if (page >= 0 && page < p.n_pages)
                        slot_row = (((int64_t)page * p.heads[1]) << p.page_log2) + (pos & ((1 << p.page_log2) - 1));
                    else if (lane == 0)
                        raise_status(p.ws, kStatBadPage);
                }
            }
            if (p.rot == 0) return;
            float cs[kOwn], sn[kOwn];
#pragma unroll
            for (int e = 0; e < kOwn; ++e) {
                const int x = p.positions ? __ldg(p.positions + (size_t)t * p.n_axes + axis[e]) : pos;
                const int f = (int)((turn[e] * (uint64_t)(int64_t)x) >> 32);             // in 2^-32 turns
                sincospif((float)f * 0x1p-31f, &sn[e], &cs[e]);
                sn[e] *= p.amplitude;
                cs[e] *= p.amplitude;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                at.c[e] = __shfl_sync(0xffffffffu, cs[e % kOwn], e / kOwn * kLanes + at.part);
                at.s[e] = __shfl_sync(0xffffffffu, sn[e % kOwn], e / kOwn * kLanes + at.part);
            }
        };
        auto sum = [](float a, float b) { return a + b; };
#pragma unroll 1
        for (int c = p.parts == 1 ? 0 : (int)((uint32_t)task % (uint32_t)p.parts); c < chunks; c += p.parts) {
            float wa[4], wb[4];
            if (MODE == kRows || c < q_chunks) {
                // ---------------- 8 vectors of q's heads (or of k's, without a cache)
                const int which = MODE == kRows && c >= q_chunks ? 1 : 0;
                const int h0 = (which ? c - q_chunks : c) * kVecs * kHeads + at.sub, heads = p.heads[which];
                const uint16_t* src = p.src[which] + (int64_t)t * p.src_stride[which];
                const bool norm = p.w[which] != nullptr;
                uint32_t w[kVecs][4];
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0u;
                    if (h0 + i * kHeads < heads) at.load(src + (int64_t)(h0 + i * kHeads) * HD, w[i]);
                }
                if (norm) at.weights(p.w[which], p.w_dtype, wa, wb);
                if (!known) look();
                if (!in) break;
                float r = 1.f;
                if (norm) {
                    float sq[kVecs];
#pragma unroll
                    for (int i = 0; i < kVecs; ++i) {
                        float a[4], b[4];
                        P::split(w[i], a, b);
                        sq[i] = 0.f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) sq[i] = fmaf(b[e], b[e], fmaf(a[e], a[e], sq[i]));
                    }
                    r = __frsqrt_rn(fmaf(join_rows<kVecs, kLanes>(sq, at.part, sum), 1.f / HD, p.eps));
                }
                uint16_t* out = p.out[which] + (int64_t)t * p.out_stride[which];
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    float a[4], b[4];
                    const float ri = norm ? __shfl_sync(0xffffffffu, r, at.sub * kLanes + i * (kLanes / kVecs)) : 1.f;
                    at.turn(w[i], norm, ri, wa, wb, a, b);
                    if (h0 + i * kHeads < heads) at.store(out + (int64_t)(h0 + i * kHeads) * HD, a, b);
                }
            } else {
                // ---------------- 4 vectors of k's heads and of v's, into the cache
                constexpr int N = kVecs / 2;
                const int h0 = (c - q_chunks) * N * kHeads + at.sub, heads = p.heads[1];
                const uint16_t* ks = p.src[1] + (int64_t)t * p.src_stride[1];
                const uint16_t* vs = p.src[2] + (int64_t)t * p.src_stride[2];
                const bool norm = p.w[1] != nullptr;
                uint32_t w[N][4];
                uint4 v[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int h = h0 + i * kHeads;
                    w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0u;
                    v[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (h >= heads) continue;
                    at.load(ks + (int64_t)h * HD, w[i]);
                    v[i] = __ldcs(reinterpret_cast<const uint4*>(vs + (int64_t)h * HD + at.part * 8));
                }
                if (norm) at.weights(p.w[1], p.w_dtype, wa, wb);
                if (!known) look();
                if (!in) break;
                float r = 1.f;
                if (norm) {
                    float sq[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        float a[4], b[4];
                        P::split(w[i], a, b);
                        sq[i] = 0.f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) sq[i] = fmaf(b[e], b[e], fmaf(a[e], a[e], sq[i]));
                    }
                    r = __frsqrt_rn(fmaf(join_rows<N, kLanes>(sq, at.part, sum), 1.f / HD, p.eps));
                }
                float a[N][4], b[N][4];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float ri = norm ? __shfl_sync(0xffffffffu, r, at.sub * kLanes + i * (kLanes / N)) : 1.f;
                    at.turn(w[i], norm, ri, wa, wb, a[i], b[i]);
                    if (p.out[1] && h0 + i * kHeads < heads)
                        at.store(p.out[1] + (int64_t)t * p.out_stride[1] + (int64_t)(h0 + i * kHeads) * HD, a[i], b[i]);
                }
                if (slot_row < 0) continue;
                if (MODE == kAppendBf16) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int h = h0 + i * kHeads;
                        if (h >= heads) continue;
                        const int64_t row = slot_row + ((int64_t)h << p.page_log2);
                        at.store(reinterpret_cast<uint16_t*>(p.dst[0]) + row * HD, a[i], b[i]);
                        *reinterpret_cast<uint4*>(p.dst[1] + (row * HD + at.part * 8) * 2) = v[i];
                    }
                } else {
                    // the rows' largest magnitudes (as bits, which order a NaN above
                    // infinity), one scale and one reciprocal per row
                    float m[kVecs];
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        uint32_t x = 0u, y = 0u;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x = max(x, max(__float_as_uint(a[i][e]) & 0x7FFFFFFFu, __float_as_uint(b[i][e]) & 0x7FFFFFFFu));
                            const uint32_t u = e == 0 ? v[i].x : (e == 1 ? v[i].y : (e == 2 ? v[i].z : v[i].w));
                            y = __vmaxu2(y, u & 0x7FFF7FFFu);
                        }
                        m[i] = __uint_as_float(x);
                        m[N + i] = __uint_as_float(max(y & 0xFFFFu, y >> 16) << 16);
                    }
                    const float big = join_rows<kVecs, kLanes>(m, at.part, [](float x, float y) {
                        return __uint_as_float(max(__float_as_uint(x), __float_as_uint(y)));
                    });
                    float inv = 0.f;
                    {
                        const int i = at.part / (kLanes / kVecs), kv = i / N, h = h0 + (i % N) * kHeads;
                        if (at.part % (kLanes / kVecs) == 0 && h < heads)
                            p.scale[kv][slot_row + ((int64_t)h << p.page_log2)] = __fdiv_rn(big, 448.f);
                        // below 2^-100 the reciprocal would overflow float32: such rows (a
                        // negative sign marks them) are scaled up by 2^64 first; rows that are
                        // zero or not finite get codes of zero
                        if (big > 0.f && big < INFINITY)
                            inv = big < kTiny ? -__fdiv_rn(448.f, big * 0x1p64f) : __fdiv_rn(448.f, big);
                    }
                    const bool as_given = !norm && p.rot == 0;   // k as it came: its midpoints count, as v's do
#pragma unroll
                    for (int i = 0; i < kVecs; ++i) {
                        const int h = h0 + (i % N) * kHeads;
                        const float f = __shfl_sync(0xffffffffu, inv, at.sub * kLanes + i * (kLanes / kVecs));
                        const float up = f < 0.f ? 0x1p64f : 1.f;
                        const uint64_t up2 = pack2(up, up), f2 = pack2(fabsf(f), fabsf(f));
                        if (h >= heads) continue;
                        const int64_t row = (slot_row + ((int64_t)h << p.page_log2)) * HD;
                        if (i >= N) {
                            const uint32_t in4[4] = {v[i % N].x, v[i % N].y, v[i % N].z, v[i % N].w};
                            uint32_t q[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) q[e] = quantise2(mul2x(pack2(lo16(in4[e]), hi16(in4[e])), up2), f2);
                            uint2 code = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
                            if (f == 0.f) code = make_uint2(0u, 0u);
                            *reinterpret_cast<uint2*>(p.dst[1] + row + at.part * 8) = code;
                        } else {
                            // float32 values: their quotient is rounded to e4m3 as it stands
                            float (&x)[4] = a[i];
                            float (&y)[4] = b[i];
                            auto two = [&](float g, float h2) {
                                const uint64_t u = mul2x(pack2(g, h2), up2);
                                if (as_given) return quantise2(u, f2);
                                float2 z;
                                unpack2(mul2x(u, f2), z.x, z.y);
                                return (uint32_t)__nv_cvt_float2_to_fp8x2(z, __NV_SATFINITE, __NV_E4M3);
                            };
                            uint32_t c0, c1;
                            if (kPairs) {
                                c0 = two(x[0], y[0]) | two(x[1], y[1]) << 16;
                                c1 = two(x[2], y[2]) | two(x[3], y[3]) << 16;
                            } else {
                                c0 = two(x[0], x[1]) | two(x[2], x[3]) << 16;
                                c1 = two(y[0], y[1]) | two(y[2], y[3]) << 16;
                            }
                            if (f == 0.f) c0 = c1 = 0u;
                            *reinterpret_cast<uint32_t*>(p.dst[0] + row + at.o0) = c0;
                            *reinterpret_cast<uint32_t*>(p.dst[0] + row + at.o1) = c1;
                        }
                    }
                }
            }
        }
    }
}

// inv_freq / 2 pi, whole turns taken off, in 2^-64 turns (a negative frequency's
// modulo 2^64).
uint64_t turns_of(double inv_freq) {
    double x = std::fabs(inv_freq) / 6.283185307179586476925;
    x -= std::floor(x);                                       // exact
    const uint64_t n = (uint64_t)std::ldexp(x, 64);
    return inv_freq < 0 ? 0 - n : n;
}

template <int HD, int MODE>
cudaError_t launch(const RopeParams& p, bool pairs, int grid, cudaStream_t s) {
    return pairs ? launch_kernel(rope_kernel<HD, true, MODE>, dim3(grid), dim3(kWarps * 32), 0, s, false, p)
                 : launch_kernel(rope_kernel<HD, false, MODE>, dim3(grid), dim3(kWarps * 32), 0, s, false, p);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
    RopeParams p = {};
    const void* src[3] = {a.q, a.k, a.v};
    const int64_t ss[3] = {a.q_stride, a.k_stride, a.v_stride};
    for (int i = 0; i < 3; ++i) {
        p.src[i] = static_cast<const uint16_t*>(src[i]);
        p.src_stride[i] = ss[i];
    }
    p.out[0] = static_cast<uint16_t*>(a.q_out);
    p.out[1] = static_cast<uint16_t*>(a.k_out);
    p.out_stride[0] = a.q_out_stride;
    p.out_stride[1] = a.k_out_stride;
    p.heads[0] = a.n_heads;
    p.heads[1] = a.n_kv_heads;
    if (a.norm) {
        p.w[0] = a.norm->q_w;
        p.w[1] = a.norm->k_w;
        p.w_dtype = a.norm->w_dtype;
        p.eps = a.norm->eps;
    }
    p.positions = a.positions;
    p.T = a.T;
    bool pairs = false;
    if (a.rope) {
        p.rot = a.rope->rot;
        p.n_axes = a.rope->n_axes;
        p.amplitude = a.rope->amplitude;
        pairs = a.rope->interleaved != 0;
        for (int i = 0; i < a.rope->rot / 2; ++i) {
            p.turn[i] = turns_of(a.rope->inv_freq[i]);
            p.axis[i] = a.rope->axis[i];
        }
    }
    int mode = kRows;
    if (a.cache) {
        const dspark_kv_cache_t& c = *a.cache;
        mode = c.dtype == DSPARK_E4M3 ? kAppendE4m3 : kAppendBf16;
        p.dst[0] = static_cast<uint8_t*>(c.k);
        p.dst[1] = static_cast<uint8_t*>(c.v);
        p.scale[0] = c.k_scale;
        p.scale[1] = c.v_scale;
        p.q_off = a.batch->q_off;
        p.kv_len = a.batch->kv_len;
        p.page_table = a.batch->page_table;
        p.ws = a.ws;
        p.R = a.batch->R;
        p.max_pages = a.batch->max_pages;
        p.n_pages = c.n_pages;
        p.page_log2 = ceil_log2_i(c.page);
    }
    // A warp per token where that fills the device; with fewer tokens their chunks
    // are spread over more warps, which work the angles out again.
    const int heads = 256 / a.head_dim;                       // heads of a vector
    const int kv_step = (mode == kRows ? kVecs : kVecs / 2) * heads;
    const int chunks = (a.n_heads + kVecs * heads - 1) / (kVecs * heads) + (a.n_kv_heads + kv_step - 1) / kv_step;
    const int64_t full = (int64_t)num_sms() * 16;
    p.parts = (int)std::min((int64_t)chunks, std::max((int64_t)1, full / a.T));
    const int64_t ctas = ((int64_t)a.T * p.parts + kWarps - 1) / kWarps;
    const int grid = (int)std::min(ctas, (int64_t)num_sms() * 16);
    const int name = mode == kRows ? kPQkRope : kPRopeWrite;
    prof_begin(name, s);
    cudaError_t e;
    if (a.head_dim == 64)
        e = mode == kRows ? launch<64, kRows>(p, pairs, grid, s)
                          : (mode == kAppendBf16 ? launch<64, kAppendBf16>(p, pairs, grid, s) : launch<64, kAppendE4m3>(p, pairs, grid, s));
    else
        e = mode == kRows ? launch<128, kRows>(p, pairs, grid, s)
                          : (mode == kAppendBf16 ? launch<128, kAppendBf16>(p, pairs, grid, s) : launch<128, kAppendE4m3>(p, pairs, grid, s));
    prof_end(s);
    return e;
}

}  // namespace dspark
