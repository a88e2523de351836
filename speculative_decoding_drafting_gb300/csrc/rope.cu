// rope.cu -- query and key heads normed and turned to their positions, packed
// rows in and out, or keys and values on into the paged cache.
//
// A head x of head_dim values becomes y = x w / sqrt(mean x^2 + eps) (where there
// is a norm), and its first `rot` values are turned in pairs (a, b):
//   a' = a cos t - b sin t,  b' = b cos t + a sin t,  t = position x inv_freq
// The turns of a position are the fraction of position x (inv_freq / 2 pi).  The
// frequency in units of 2^-64 turns is rounded once, to 53 bits; its product with the
// position in 64-bit integers loses whole turns and nothing else, however far the
// position.  Cosine and sine of the fraction are float32, and everything up to the
// one rounding of a stored value is float32.
//
// Bound by the bytes: each value is read and written once.  Lanes hold 8 values
// of a head, 4 and the 4 that they are turned with, so that neither a shuffle
// nor a second load is needed; 16 lanes share a head of 128 (8 one of 64).  A CTA
// takes up to 4 tokens together: their requests and places are looked up by the
// lanes of one warp, their angles worked out by all threads, once for all heads,
// and kept in shared memory.  Then each warp goes through tasks of 4 vectors of 32
// lanes, in packed float32 arithmetic; the other warps of the SM cover its loads.
// Measured (GB300, against 6.68 TB/s of a plain copy): 23457 tokens of 28 + 4 heads
// of 128, three axes, no norm, 63 us, 6.1 TB/s; 41925 tokens of 32 + 8 + 8 heads with
// norms into an e4m3 cache, the keys also as rows, 189 us, 5.5 TB/s; into a bf16 one
// 182 to 188 us, 5.9 to 6.1 TB/s.  (A warp per token, with its own look-up and angles,
// 8 vectors at a time and one value per instruction: 75, 190 and 187, and 91 for 76
// with norms.  A float32 value per instruction in the present form: 87 with norms, 209
// into e4m3.)
#include <algorithm>
#include <cmath>

#include "kernels.h"
#include "kv.cuh"
#include "profile.h"
#include "sm100.cuh"

namespace dspark {

namespace {

constexpr int kWarps = 4;
constexpr int kVecs = 4;               // vectors of a task: of q's or k's heads, or 2 of k's and 2 of v's
constexpr int kToks = 4;               // tokens of a CTA at most (8: 68 us for 64)
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
    int T, toks;                       // toks: tokens of a CTA
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
    // The pairs' first and second values, two and two (one instruction for both).
    __device__ __forceinline__ static void split(const uint32_t (&w)[4], uint64_t (&a)[2], uint64_t (&b)[2]) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (kPairs) {
                a[e] = pack2(lo16(w[2 * e]), lo16(w[2 * e + 1]));
                b[e] = pack2(hi16(w[2 * e]), hi16(w[2 * e + 1]));
            } else {
                a[e] = pack2(lo16(w[e]), hi16(w[e]));
                b[e] = pack2(lo16(w[2 + e]), hi16(w[2 + e]));
            }
        }
    }
    __device__ __forceinline__ static float squares(const uint32_t (&w)[4]) {
        uint64_t a[2], b[2];
        split(w, a, b);
        float x, y;
        unpack2(fma2(b[1], b[1], fma2(b[0], b[0], fma2(a[1], a[1], mul2x(a[0], a[0])))), x, y);
        return x + y;
    }
    // a head's values times r and the weights
    __device__ __forceinline__ static void norm(uint64_t (&a)[2], uint64_t (&b)[2], float r, const uint64_t (&wa)[2],
                                                const uint64_t (&wb)[2]) {
        const uint64_t r2 = pack2(r, r);
#pragma unroll
        for (int e = 0; e < 2; ++e) a[e] = mul2x(a[e], mul2x(r2, wa[e])), b[e] = mul2x(b[e], mul2x(r2, wb[e]));
    }
    // turned by the cosines, sines and negative sines of the lane's four angles
    __device__ __forceinline__ void turn(uint64_t (&a)[2], uint64_t (&b)[2], const uint64_t (&c)[2], const uint64_t (&s)[2],
                                         const uint64_t (&minus_s)[2]) const {
        if (!turns) return;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint64_t x = a[e], y = b[e];
            a[e] = fma2(x, c[e], mul2x(y, minus_s[e]));
            b[e] = fma2(y, c[e], mul2x(x, s[e]));
        }
    }
    // as float32 in the order of the row: o0 .. o0 + 3, then o1 .. o1 + 3
    __device__ __forceinline__ static void in_order(const uint64_t (&a)[2], const uint64_t (&b)[2], float (&x)[8]) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (kPairs) {
                unpack2(a[e], x[4 * e], x[4 * e + 2]);
                unpack2(b[e], x[4 * e + 1], x[4 * e + 3]);
            } else {
                unpack2(a[e], x[2 * e], x[2 * e + 1]);
                unpack2(b[e], x[4 + 2 * e], x[5 + 2 * e]);
            }
        }
    }
    __device__ __forceinline__ void store(uint16_t* row, const uint64_t (&a)[2], const uint64_t (&b)[2]) const {
        float x[8];
        in_order(a, b, x);
        const uint2 u = make_uint2(two_bf16(x[0], x[1]), two_bf16(x[2], x[3])), v = make_uint2(two_bf16(x[4], x[5]), two_bf16(x[6], x[7]));
        if (kPairs) {
            *reinterpret_cast<uint4*>(row + o0) = make_uint4(u.x, u.y, v.x, v.y);
        } else {
            *reinterpret_cast<uint2*>(row + o0) = u;
            *reinterpret_cast<uint2*>(row + o1) = v;
        }
    }
    __device__ __forceinline__ void weights(const void* w, int dtype, uint64_t (&a)[2], uint64_t (&b)[2]) const {
        if (dtype == DSPARK_F32) {
            const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + o0));
            const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + o1));
            a[0] = kPairs ? pack2(u.x, u.z) : pack2(u.x, u.y);
            a[1] = kPairs ? pack2(v.x, v.z) : pack2(u.z, u.w);
            b[0] = kPairs ? pack2(u.y, u.w) : pack2(v.x, v.y);
            b[1] = kPairs ? pack2(v.y, v.w) : pack2(v.z, v.w);
        } else {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + o0));
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + o1));
            const uint32_t x[4] = {u.x, u.y, v.x, v.y};
            split(x, a, b);
        }
    }
};

// What a CTA knows of one of its tokens.
struct Token {
    int64_t row;                       // of head 0 in the cache, in units of a head's rows (negative: no place)
    int pos;                           // place in its request
    int in;                            // whether it belongs to one
};

// The tokens [t0, t0 + n) (n <= kToks) by one warp, a lane for each.
__device__ __forceinline__ void look_up(const RopeParams& p, int t0, int n, Token* out) {
    const int lane = threadIdx.x & 31, t = t0 + min(lane, n - 1);
    const int64_t most = (int64_t)p.max_pages << p.page_log2;
    // the first token's request, and how many begin up to each of the others
    const int r0 = find_request(p.q_off, p.R, t0);
    const int begins = r0 + 1 + lane < p.R ? __ldg(p.q_off + r0 + 1 + lane) : 0x7FFFFFFF;
    int r = r0;
#pragma unroll 1
    for (int i = 1; i < n; ++i) {
        const uint32_t m = __ballot_sync(0xffffffffu, begins <= t0 + i);
        // all 32 have begun: many of them empty
        const int ri = m == 0xFFFFFFFFu ? find_request(p.q_off, p.R, t0 + i) : r0 + __popc(m);
        if (lane == i) r = ri;
    }
    if (lane >= n) return;
    const RowRange rows = row_range(p.q_off, r, p.T);
    Token k;
    k.in = t >= rows.a && t < rows.b;
    k.pos = clamped_len(p.kv_len, r, most) - (rows.b - t);
    k.row = -1;
    if (k.in && k.pos >= 0 && p.heads[1] > 0) {
        const int page = __ldg(p.page_table + (size_t)r * p.max_pages + (k.pos >> p.page_log2));
        if (page >= 0 && page < p.n_pages)
            k.row = (((int64_t)page * p.heads[1]) << p.page_log2) + (k.pos & ((1 << p.page_log2) - 1));
        else
            raise_status(p.ws, kStatBadPage);
    }
    out[lane] = k;
}

template <int HD, bool kPairs, int MODE>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const __grid_constant__ RopeParams p) {
    using P = Place<HD, kPairs>;
    constexpr int kLanes = P::kLanes, kHeads = P::kHeads, kHalf = HD / 2;
    constexpr int kStep = kVecs * kHeads;                     // heads of a task
    // whether the next task's loads are issued before this one's work: it takes
    // registers, and pays where there is much of it (41925 tokens into an e4m3 cache 195
    // -> 189 us; rows with a norm 70 -> 74, without one 63 -> 64)
    constexpr bool kAhead = MODE == kAppendE4m3;
    __shared__ __align__(16) float cosines[kToks][kHalf], sines[kToks][kHalf];
    __shared__ Token tokens[kToks];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const P at(lane, p.rot);
    if (MODE != kRows && blockIdx.x == gridDim.x - 1)
        check_requests(p.q_off, p.kv_len, p.R, p.T, (int64_t)p.max_pages << p.page_log2, p.ws);

    const int t0 = blockIdx.x * p.toks, n = min(p.toks, p.T - t0);
    // a token's tasks: heads of q, then heads of k, or 2 vectors of k's heads and 2 of v's
    constexpr int kKvStep = MODE == kRows ? kStep : kStep / 2;
    const int first_kv = (p.heads[0] + kStep - 1) / kStep, per = first_kv + (p.heads[1] + kKvStep - 1) / kKvStep;
    // task c's vectors of token i (heads that are not there are not loaded: their lanes
    // work on what the registers hold and store nothing)
    auto load = [&](int i, int c, uint32_t (&w)[kVecs][4]) {
        const int64_t t = t0 + i;
        const bool kv = c >= first_kv;
        const int h0 = kv ? (c - first_kv) * kKvStep : c * kStep, heads = kv ? p.heads[1] : p.heads[0];
        const uint16_t* row = (kv ? p.src[1] + t * p.src_stride[1] : p.src[0] + t * p.src_stride[0]) + (h0 + at.sub) * HD;
        const uint16_t* vrow = MODE == kRows ? nullptr : p.src[2] + t * p.src_stride[2] + (h0 + at.sub) * HD + at.part * 8;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            if (MODE != kRows && kv && v >= kVecs / 2) {
                if (h0 + (v - kVecs / 2) * kHeads + at.sub >= heads) continue;
                const uint4 x = __ldcs(reinterpret_cast<const uint4*>(vrow + (v - kVecs / 2) * (kHeads * HD)));
                w[v][0] = x.x, w[v][1] = x.y, w[v][2] = x.z, w[v][3] = x.w;
            } else if (h0 + v * kHeads + at.sub < heads) {
                at.load(row + v * (kHeads * HD), w[v]);
            }
        }
    };
    // where a warp is: token i of the CTA, task c of it
    int i = 0, c = warp;
    auto settle = [&]() {
        while (c >= per) c -= per, ++i;
    };
    settle();
    uint32_t w[kVecs][4];
    if (i < n) load(i, c, w);

    // the tokens' places and angles, while the first loads are in flight
    if (MODE != kRows) {
        if (warp == 0) look_up(p, t0, n, tokens);
        __syncthreads();
    }
    if (p.rot > 0) {
        const int f = threadIdx.x % kHalf;
        const uint64_t turn = p.turn[f];
        const int axis = p.axis[f];
        if (f < p.rot / 2) {
            for (int k = threadIdx.x / kHalf; k < n; k += kWarps * 32 / kHalf) {
                const int x = p.positions ? __ldg(p.positions + (int64_t)(t0 + k) * p.n_axes + axis)
                                          : (MODE == kRows ? 0 : tokens[k].pos);
                // of a turn, in 2^-32: the nearest quarter, and what is left of it, whose float32
                // is off by 2^-28 turns at most (that of the whole by 2^-26)
                const uint32_t part = (uint32_t)((turn * (uint64_t)(int64_t)x) >> 32), quarter = (part + (1u << 29)) >> 30;
                float u, v;
                sincospif((float)(int)(part - (quarter << 30)) * 0x1p-31f, &v, &u);
                float cs = quarter & 1u ? -v : u, sn = quarter & 1u ? u : v;
                if (quarter & 2u) cs = -cs, sn = -sn;
                cosines[k][f] = cs * p.amplitude;
                sines[k][f] = sn * p.amplitude;
            }
        }
        __syncthreads();
    }
    auto sum = [](float a, float b) { return a + b; };
#pragma unroll 1
    while (i < n) {
        const int ti = i, tc = c;
        const int64_t t = t0 + ti;
        c += kWarps;
        settle();
        uint32_t next[kVecs][4];
        if (kAhead && i < n) load(i, c, next);
        uint64_t cs[2], sn[2], minus_sn[2];
        if (at.turns) {
            const float4 x = *reinterpret_cast<const float4*>(&cosines[ti][at.part * 4]), y = *reinterpret_cast<const float4*>(&sines[ti][at.part * 4]);
            cs[0] = pack2(x.x, x.y), cs[1] = pack2(x.z, x.w);
            sn[0] = pack2(y.x, y.y), sn[1] = pack2(y.z, y.w);
            minus_sn[0] = pack2(-y.x, -y.y), minus_sn[1] = pack2(-y.z, -y.w);
        }
        const bool in = MODE == kRows || tokens[ti].in;
        const bool kv = tc >= first_kv;
        const void* weights = kv ? p.w[1] : p.w[0];
        uint64_t wa[2], wb[2];
        if (weights) at.weights(weights, p.w_dtype, wa, wb);
        if (in && (MODE == kRows || !kv)) {
            // ---------------- heads of q (or of k, without a cache)
            const int h0 = (kv ? tc - first_kv : tc) * kStep, heads = kv ? p.heads[1] : p.heads[0];
            float r = 1.f;
            if (weights) {
                float sq[kVecs];
#pragma unroll
                for (int v = 0; v < kVecs; ++v) sq[v] = P::squares(w[v]);
                r = __frsqrt_rn(fmaf(join_rows<kVecs, kLanes>(sq, at.part, sum), 1.f / HD, p.eps));
            }
            uint16_t* row = (kv ? p.out[1] + t * p.out_stride[1] : p.out[0] + t * p.out_stride[0]) + (h0 + at.sub) * HD;
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                if (h0 + v * kHeads >= heads) break;
                uint64_t a[2], b[2];
                P::split(w[v], a, b);
                if (weights) P::norm(a, b, __shfl_sync(0xffffffffu, r, at.sub * kLanes + v * (kLanes / kVecs)), wa, wb);
                at.turn(a, b, cs, sn, minus_sn);
                if (h0 + v * kHeads + at.sub < heads) at.store(row + v * (kHeads * HD), a, b);
            }
        } else if (in) {
            // ---------------- heads of k and v, into the cache
            constexpr int N = kVecs / 2;
            const int h0 = (tc - first_kv) * kKvStep + at.sub, heads = p.heads[1];
            const int64_t slot = tokens[ti].row;
            uint64_t a[N][2], b[N][2];
            float r = 1.f;
            if (weights) {
                float sq[N];
#pragma unroll
                for (int v = 0; v < N; ++v) sq[v] = P::squares(w[v]);
                r = __frsqrt_rn(fmaf(join_rows<N, kLanes>(sq, at.part, sum), 1.f / HD, p.eps));
            }
#pragma unroll
            for (int v = 0; v < N; ++v) {
                P::split(w[v], a[v], b[v]);
                if (weights) P::norm(a[v], b[v], __shfl_sync(0xffffffffu, r, at.sub * kLanes + v * (kLanes / N)), wa, wb);
                at.turn(a[v], b[v], cs, sn, minus_sn);
                if (p.out[1] && h0 + v * kHeads < heads)
                    at.store(p.out[1] + t * p.out_stride[1] + (h0 + v * kHeads) * HD, a[v], b[v]);
            }
            if (slot >= 0 && MODE == kAppendBf16) {
#pragma unroll
                for (int v = 0; v < N; ++v) {
                    const int h = h0 + v * kHeads;
                    if (h >= heads) continue;
                    const int64_t row = (slot + ((int64_t)h << p.page_log2)) * HD;
                    at.store(reinterpret_cast<uint16_t*>(p.dst[0]) + row, a[v], b[v]);
                    *reinterpret_cast<uint4*>(p.dst[1] + (row + at.part * 8) * 2) = make_uint4(w[N + v][0], w[N + v][1], w[N + v][2], w[N + v][3]);
                }
            }
            if (slot >= 0 && MODE == kAppendE4m3) {
                // the rows' largest magnitudes (as bits, which order a NaN above
                // infinity), one scale and one reciprocal per row
                float m[kVecs], x[N][8];
#pragma unroll
                for (int v = 0; v < N; ++v) {
                    P::in_order(a[v], b[v], x[v]);
                    uint32_t most = 0u, y = 0u;
#pragma unroll
                    for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(x[v][e]) & 0x7FFFFFFFu);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y = __vmaxu2(y, w[N + v][e] & 0x7FFF7FFFu);
                    m[v] = __uint_as_float(most);
                    m[N + v] = __uint_as_float(max(y & 0xFFFFu, y >> 16) << 16);
                }
                const float big = join_rows<kVecs, kLanes>(m, at.part, [](float x, float y) {
                    return __uint_as_float(max(__float_as_uint(x), __float_as_uint(y)));
                });
                // 448 / big as inv + rest, to about 48 bits: a quotient is then rounded once, so
                // that where a turn by 0 leaves a row's bf16 values as they came their
                // midpoints are ties, as v's are (one product with inv took the wrong
                // side of 5 times as many as a division)
                float inv = 0.f, rest = 0.f;
                {
                    constexpr int kOwn = kLanes / kVecs;      // lanes that hold a row's largest
                    const int v = at.part / kOwn, kv = v / N, h = h0 + v % N * kHeads;
                    if (at.part % kOwn == 0 && h < heads) p.scale[kv][slot + ((int64_t)h << p.page_log2)] = __fdiv_rn(big, 448.f);
                    // below 2^-100 the reciprocal would overflow float32: such rows (a
                    // negative sign marks them) are scaled up by 2^64 first; rows that are
                    // zero or not finite get codes of zero
                    if (big > 0.f && big < INFINITY) {
                        const float a = big < kTiny ? big * 0x1p64f : big;
                        inv = __fdiv_rn(448.f, a);
                        rest = fmaf(-inv, a, 448.f) * inv * (1.f / 448.f);
                        if (big < kTiny) inv = -inv;
                    }
                }
#pragma unroll
                for (int v = 0; v < kVecs; ++v) {
                    const int h = h0 + v % N * kHeads;
                    const float f = __shfl_sync(0xffffffffu, inv, at.sub * kLanes + v * (kLanes / kVecs));
                    const float lo = v < N ? __shfl_sync(0xffffffffu, rest, at.sub * kLanes + v * (kLanes / kVecs)) : 0.f;
                    const float up = f < 0.f ? 0x1p64f : 1.f;
                    const uint64_t up2 = pack2(up, up), f2 = pack2(fabsf(f), fabsf(f)), lo2 = pack2(lo, lo);
                    if (h >= heads) continue;
                    const int64_t row = (slot + ((int64_t)h << p.page_log2)) * HD;
                    if (v >= N) {
                        uint32_t q[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) q[e] = quantise2(mul2x(pack2(lo16(w[v][e]), hi16(w[v][e])), up2), f2);
                        uint2 code = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
                        if (f == 0.f) code = make_uint2(0u, 0u);
                        *reinterpret_cast<uint2*>(p.dst[1] + row + at.part * 8) = code;
                    } else {
                        auto two = [&](float g, float h2) {
                            const uint64_t u = mul2x(pack2(g, h2), up2);
                            float2 z;
                            unpack2(fma2(u, f2, mul2x(u, lo2)), z.x, z.y);
                            return (uint32_t)__nv_cvt_float2_to_fp8x2(z, __NV_SATFINITE, __NV_E4M3);
                        };
                        const float (&y)[8] = x[v % N];
                        uint32_t c0 = two(y[0], y[1]) | two(y[2], y[3]) << 16, c1 = two(y[4], y[5]) | two(y[6], y[7]) << 16;
                        if (f == 0.f) c0 = c1 = 0u;
                        *reinterpret_cast<uint32_t*>(p.dst[0] + row + at.o0) = c0;
                        *reinterpret_cast<uint32_t*>(p.dst[0] + row + at.o1) = c1;
                    }
                }
            }
        }
        if (kAhead) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
#pragma unroll
                for (int e = 0; e < 4; ++e) w[v][e] = next[v][e];
        } else if (i < n) {
            load(i, c, w);
        }
    }
}

// inv_freq / 2 pi, whole turns taken off, in 2^-64 turns (a negative frequency's
// modulo 2^64).
uint64_t turns_of(double inv_freq) {
    double x = std::fabs(inv_freq) / 6.283185307179586476925;
    x -= std::floor(x);                                       // exact
    const uint64_t n = (uint64_t)(x * 0x1p64);
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
    // Tokens share a CTA where there are enough of them to fill the device (about 6
    // CTAs an SM) all the same.
    p.toks = (int)std::min((int64_t)kToks, std::max((int64_t)1, (int64_t)a.T / (num_sms() * 6)));
    const int grid = (a.T - 1) / p.toks + 1;
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
