// attn_paged.cu -- attention of each request's newest tokens over its paged
// cache (sm_103a: TMA, tcgen05, TMEM).
//
// For the rows (new token x query heads of one key-value head's group) of a
// row tile and a tile of 128 keys the kernel computes, transposed,
//   S^T = K Q^T     [128 keys x rows]      A = K tile (K-major), B = Q
//   P^T = 2^(S^T c - m)                    c = scale log2(e), m = the rows' reference
//   O^T += V^T P^T  [head_dim x rows]      A = V tile as it lies (MN-major), B = P^T
// so that the long axis (keys, then head_dim) fills the tensor core's 128
// rows and the few query rows are its N, 16 to 64: one request's block of
// gamma + 1 tokens costs one pass over its keys, whatever the group.  It is
// bound by the cache's bytes: 64 KB of bf16 per key tile take the SM about
// 2800 cycles at the measured copy rate, its two products under 600.
// Measured (GB300, against 6.68 TB/s of a plain copy): 256 requests of 200 to
// 4000 keys, blocks of 1 to 6 tokens, 32 heads over 8 of 128, bf16: 330 to 335
// us, 6.7 TB/s; 64 requests of 500 to 8000 e4m3 keys, one token, 64 heads over 8:
// 113 us, 5.1 TB/s (5.6 TB/s at 8192 keys each); two requests of 150001 and
// 260001 e4m3 keys at most, blocks of 6, 32 heads over 4: 138 us, 3.8 TB/s.
//
// One persistent CTA per SM walks an equal span of the line of all items' key
// tiles (attn_plan.h); pieces of split items go to the workspace and a second
// launch joins them in a fixed order.  (Counters that let the last CTA of an
// item join it would save that launch, but need a workspace that starts at
// zero; only its status word does.)  The kernel starts beside the end of the
// one before it: barriers, tensor memory and descriptors are ready by then.
//
//   warp 0      K tiles by TMA, page by page (a page id out of range lies past
//               the tensor's end, so it reads as zeros), and e4m3 scales
//   warp 1      the scores' MMAs
//   warp 2      the list of this CTA's segments, a few ahead of the others, and
//               V tiles by TMA
//   warp 3      the products' MMAs
//   warps 4-19  four softmax units of four warps.  Items of up to 32 rows go
//               through four streams of key tiles (unit u takes every fourth),
//               wider ones through two streams of two units with half the rows
//               each, each stream with its own references, sums and
//               accumulator, so that some exponentiate while the products of
//               others run.  Thread = key, registers = rows.  The reference of
//               a row is raised only when a score exceeds it by more than 8
//               binary orders (a vote per tile; weights up to 2^8 are far
//               inside bf16 and float32; 5.5 orders above the lift for e4m3), so
//               a tile costs no maximum over its keys.
//   warps 20-23 bring the next segment's Q rows, then join the streams of the
//               finished one and store it, while the units are at the next
//               (accumulators alternate)
// The loops are kept short, and what runs once per segment is a function of
// its own: 24 warps of different code share one instruction cache.
//
// e4m3 caches: K tiles go to the tensor core as they are.  Each row of Q is
// split into 2^e (hi + lo), both e4m3, 2^e such that the row's largest value is
// in [128, 256): bf16's 8 significant bits are two times e4m3's 4, and e4m3
// holds what the first term leaves down to 2^-9, so the split is exact except
// for values below 2^-9 of the row's largest (0.25 of 128), which are off by
// half of that step, 2^-17 of the largest, at most.  hi and lo follow one another
// along K.
// V tiles are widened to fp16 (one instruction for two values) by the units
// that made the tile's weights, the one shared-memory pass that e4m3 costs.
// V's scale joins the exponent, w = 2^(score + log2 scale - m + 10), so that
// the weights, whatever the scales, lie below 2^15.5 with fp16's 11 bits down to
// 2^-24 of the row's largest; the sum takes w / scale.
//
// Keys a row must not see get weight 0 by selection, not by multiplication;
// V rows past the item's last key are zeroed in shared memory, since 0 times
// a stale NaN would be NaN.
#include <type_traits>

#include <cstddef>
#include <cuda.h>

#include "attn_plan.h"
#include "kernels.h"
#include "kv.cuh"
#include "profile.h"
#include "sm100.cuh"

namespace dspark {

namespace {

constexpr float kFloorRef = -1e30f;     // reference before any score: finite, below every score
constexpr int kUnits = 4;               // softmax units of 128 threads
constexpr int kUnitRows = 32;           // columns of S^T a unit handles

template <int HD, bool F8>
struct Cfg {
    static constexpr int kTileBytes = kKeyTile * HD * 2;                   // a K or V tile as bf16
    static constexpr int kHalves = HD / 64;                                // 128-byte swizzle atoms of a row
    static constexpr int kHalfBytes = kKeyTile * 128;
    static constexpr int kLoadBytes = F8 ? kKeyTile * HD : kTileBytes;     // a tile as it lies in the cache
    static constexpr int kK = F8 ? (HD == 128 ? 2 : 4) : (HD == 128 ? 2 : 5);       // K tiles on the way
    static constexpr int kV = F8 ? (HD == 128 ? 4 : 6) : (HD == 128 ? 3 : 5);       // V tiles
    static constexpr int kW = F8 ? (HD == 128 ? 2 : 3) : 0;                // widened V tiles
    static constexpr int kSc = F8 ? 4 : 0;                                 // scales of a tile (K, V)
    static constexpr int kScBytes = 2 * kKeyTile * 4;                      // K's scales, then V's
    static constexpr int kPBytes = kKeyTile * kUnitRows * 2;               // a unit's P^T
    // two Q places; at head_dim 128 an item of more than 32 rows takes both
    static constexpr int kQRows = HD == 128 ? 32 : 64;
    static constexpr int kQBytes = kQRows * HD * 2;                        // bf16 rows, or hi and lo
    static constexpr int kScMod = kSc ? kSc : 1;                           // divisor (unused without e4m3)
    // bits by which a weight's exponent is lifted, and may exceed that (fp16 ends
    // at 2^16; with 4 instead of 5.5 the long e4m3 case took 149 us for 138)
    static constexpr float kLift = F8 ? 10.f : 0.f, kLazy = F8 ? 5.5f : 8.f;
    static constexpr int kOffV = kK * kLoadBytes;
    static constexpr int kOffW = kOffV + kV * kLoadBytes;
    static constexpr int kOffP = kOffW + kW * kTileBytes;
    static constexpr int kOffQ = kOffP + kUnits * kPBytes;
    static constexpr int kOffSc = kOffQ + 2 * kQBytes;
    static constexpr int kOffMisc = kOffSc + kSc * kScBytes;
};
constexpr uint32_t kColO = kUnits * kUnitRows;         // TMEM: scores, two sets of accumulators, scores again
constexpr uint32_t kColS1 = 3 * kUnits * kUnitRows;
constexpr uint32_t kTmem = 512;
constexpr int kThreads = 32 * (8 + 4 * kUnits);
constexpr uint32_t kReaders = 8 + 4 * kUnits;                              // arrivals that free a segment's place
constexpr int kSegs = 8;                // segments in flight between the roles

// A segment as the roles read it from shared memory (rows = 0: the end).
struct SegInfo {
    int r, j, h;
    int t0, n, tiles;                  // key tiles [t0, t0 + n) of tiles
    int keys, rows;
    int tok, head;                     // the first row's new token and its place in the group
    int rest;                          // as in Segment
    uint32_t line;                     // key tiles of the segments before it
    uint32_t run;                      // the same for the first of the segments of equal shape that it belongs to
    int qp;                            // its Q place: 0, 1, or 2 for both
    uint32_t q_use;                    // how often place 0 (low half) and 1 have been used before
    Request q;
};

struct Bars {
    uint64_t seg_full[kSegs], seg_empty[kSegs];
    uint64_t k_full[5], k_empty[5], v_full[6], v_empty[6];
    uint64_t w_empty[3];               // widened V tiles (p_full says that one is made)
    uint64_t c_full[4], c_empty[4];    // scales
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2][kUnits], s_free[2][kUnits], p_full[kUnits], pv_done[kUnits];
    uint64_t o_done[2], l_done[2], e_free[2];   // a segment's accumulators, its sums; both read
    uint64_t r_done;                   // all products before a change of shape
    uint64_t done;
};

// How many arrivals each of them takes, in the same order.
struct BarCounts {
    uint8_t n[sizeof(Bars) / sizeof(uint64_t)];
};
template <bool F8>
constexpr BarCounts bar_counts() {
    BarCounts c = {};
    auto set = [&](size_t at, int n, int count) {
        for (int i = 0; i < n; ++i) c.n[at / sizeof(uint64_t) + i] = (uint8_t)count;
    };
    set(0, sizeof(Bars) / sizeof(uint64_t), 1);
    set(offsetof(Bars, c_full), 4, 32);
    set(offsetof(Bars, c_empty), 4, 8);
    set(offsetof(Bars, q_full), 2, 128);
    set(offsetof(Bars, q_empty), 2, F8 ? 1 + 4 * kUnits : 1);
    set(offsetof(Bars, s_free), 2 * kUnits, 4);
    set(offsetof(Bars, p_full), kUnits, 4);
    set(offsetof(Bars, seg_empty), kSegs, kReaders);
    set(offsetof(Bars, l_done), 2, 4 * kUnits);
    set(offsetof(Bars, e_free), 2, 4);
    set(offsetof(Bars, done), 1, 2);
    return c;
}
template <bool F8>
__constant__ const BarCounts kBarCounts = bar_counts<F8>();

struct alignas(16) Misc {
    SegInfo seg[kSegs];
    float ref[kUnits][kUnitRows];      // reference of a row
    float nref[kUnits][kUnitRows];     // kLift minus it
    float qm[kUnits][kUnitRows];       // 2^e of a row's split
    float fac[kUnits][kUnitRows];      // factor of a raised reference
    float red[kUnits][4][kUnitRows];   // per-warp maxima, and sums
    float q_scale[2 * kRowTile];       // 2^e of the Q places' rows
    // what a finished segment hands on, by its parity
    float fin_m[2][kUnits][kUnitRows];
    float fin_l[2][kUnits][kUnitRows];
    float join[kUnits][kUnitRows];     // factor of a stream's row
    uint8_t* row_at[kRowTile];         // a row's place in out or in the piece (null: no row)
    int64_t scan[32];
    int64_t total, start_skip;
    int start_r;
    uint32_t tmem;
    WaitState wst;
    Bars b;
};

template <int HD, bool F8>
constexpr size_t smem_bytes() {
    constexpr size_t bytes = 1024 + Cfg<HD, F8>::kOffMisc + sizeof(Misc);
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    return bytes;
}

// What a CTA tells the join about the item that its span ends inside of.
struct JoinDesc {
    int r, j, h, last;                 // r < 0: none; last: the CTA of the item's last piece
};

struct PagedParams {
    const uint16_t* q;
    int64_t q_stride;
    PlanInput plan;
    const int32_t* page_table;
    const float *k_scale, *v_scale;    // e4m3 only
    uint16_t* out;
    float* lse;
    void* ws;
    JoinDesc* desc;                    // [grid]
    float* part;                       // [grid][2] pieces: m [kRowTile], l [kRowTile], O [kRowTile][HD]
    int max_pages, n_pages, page_log2, heads;
    float scale2;                      // scale log2(e)
};

__device__ __forceinline__ size_t piece_floats(int hd) { return (size_t)kRowTile * (hd + 2); }

struct Maps {
    CUtensorMap k, v;
};

// Shared-memory operand of e4m3 rows of HD bytes: 128-byte swizzle at
// head_dim 128, 64-byte at 64.
template <int HD>
__device__ __forceinline__ uint64_t desc_f8(const void* p) {
    return HD == 128 ? smem_desc_sw128(p, 16, 1024) : smem_desc_sw64(p, 16, 512);
}
// Byte offset of 16-byte piece c of row r in that layout.
template <int HD>
__device__ __forceinline__ int swz_f8(int r, int c) {
    return r * HD + (HD == 128 ? (c ^ (r & 7)) : (c ^ ((r >> 1) & 3))) * 16;
}

// Loads that may move past stores and barriers (nothing in the kernel writes
// what they read) but, unlike the read-only path, see what the kernel before
// this one wrote while this one had started: their addresses come from data
// read after pdl_wait().
__device__ __forceinline__ uint4 load16(const void* p) {
    uint4 v;
    asm("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ int load4(const int32_t* p) {
    int v;
    asm("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// One lane's 8 values of a Q row that `LANES` lanes share: e4m3 codes of hi
// and lo with q = 2^e (hi + lo), and 2^e (NaN for a row that is not
// finite, which makes its scores NaN).
template <int LANES>
__device__ __forceinline__ float split_e4m3(uint4 v, uint2& hi, uint2& lo) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t big = max(m & 0xFFFFu, m >> 16);           // bf16 bits of the row's largest magnitude
    // 2^e: the largest value's power of two over 128, inside float32's normal range
    const int ex = min(max((int)(big >> 7) - 7, 1), 253);
    const float up = __uint_as_float((uint32_t)(254 - ex) << 23), scale = __uint_as_float((uint32_t)ex << 23);
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = bf16_bits_to_float(w[i] & 0xFFFFu) * up, b = bf16_bits_to_float(w[i] >> 16) * up;
        const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3);
        const float2 f = __half22float2(reinterpret_cast<const __half2&>(back));
        h[i] = c;
        l[i] = __nv_cvt_float2_to_fp8x2(make_float2(a - f.x, b - f.y), __NV_SATFINITE, __NV_E4M3);
    }
    hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
    return big >= 0x7F80u ? NAN : scale;
}

// The Q places of a segment: f(place, earlier uses of it) for each.
template <typename F>
__device__ __forceinline__ void q_places(const SegInfo& s, F f) {
    if (s.qp != 1) f(0, s.q_use & 0xFFFFu);
    if (s.qp != 0) f(1, s.q_use >> 16);
}

// A row tile's layout over units: width (columns of Q in use), streams.
struct Shape {
    int cols, streams;
    bool wide;
    __device__ __forceinline__ explicit Shape(int rows)
        : cols(max((rows + 15) & ~15, 16)), streams(rows > 32 ? 2 : 4), wide(rows > 32) {}
    // columns of a unit
    __device__ __forceinline__ int width() const { return wide ? cols / 2 : kUnitRows; }
    // stream of key tile i of a segment
    __device__ __forceinline__ int stream_at(const SegInfo& s, int i) const {
        return (int)((s.line - s.run + (uint32_t)i) & (uint32_t)(streams - 1));
    }
    // which of its two score tiles that stream uses for it
    __device__ __forceinline__ uint32_t turn_at(const SegInfo& s, int i) const {
        return ((s.line - s.run + (uint32_t)i) >> (wide ? 1 : 2)) & 1u;
    }
    // first TMEM column of a stream's scores, and of its accumulator in a set
    __device__ __forceinline__ uint32_t column(int stream) const { return (uint32_t)stream * (wide ? 64u : 32u); }
};

// ------------------------------------------------------------------ softmax
struct SoftState {
    uint32_t tiles;                    // key tiles this unit has taken
    uint32_t phases;                   // parity of the next wait for each of its score tiles, by bit
    uint32_t seg;                      // segments so far
};

// One segment's key tiles of unit u.  The unit's threads all
// walk the same barriers even after a wait ran out (the results are then not
// stored), so that no named barrier is left waiting.
template <int HD, bool F8, int kMost>
__device__ __forceinline__ void soft_segment(const PagedParams& p, const SegInfo& sg, Misc* M, uint8_t* smem,
                                             uint32_t tmem, int u, SoftState& st) {
    using C = Cfg<HD, F8>;
    volatile WaitState* ab = &M->wst;
    const Shape sh(sg.rows);
    const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int tr = wq * 32 + lane;                            // key of the tile; head_dim index of O^T
    // columns of this unit: a half of a wide row tile
    constexpr bool wide = kMost > kUnitRows;
    constexpr int N = wide ? kMost / 2 : kMost, streams = wide ? kUnits / 2 : kUnits;
    const int bar = 1 + u, parity = st.seg & 1;
    const int stream = wide ? u >> 1 : u, coff = wide ? (u & 1) * N : 0;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t tS0 = tmem + lanes + sh.column(stream) + (uint32_t)coff;
    const uint32_t tO = tS0 + kColO * (1 + parity);
    uint8_t* P = smem + C::kOffP + (wide ? 2 * stream : u) * C::kPBytes + (coff / 8) * (kKeyTile * 16);

    // this unit's rows (what the segment before left is no longer read)
    if (F8) q_places(sg, [&](int k, uint32_t use) { wait_bar(&M->b.q_full[k], use & 1u, ab); });
    if (tr < N) {
        M->ref[u][tr] = kFloorRef;
        M->nref[u][tr] = -kFloorRef;
        if (F8) M->qm[u][tr] = M->q_scale[(sg.qp == 1 ? C::kQRows : 0) + coff + tr];
    }
    named_sync(bar, 128);
    if (F8 && lane == 0) q_places(sg, [&](int k, uint32_t) { mbar_arrive(&M->b.q_empty[k]); });   // the row scales are copied

    float l = 0.f;                                            // this warp's sum of row `lane`
    const int lim0 = plan_token_keys(sg.q, sg.tok);           // the first row sees the fewest keys
    const int n = sg.n, t0 = sg.t0;
    const uint32_t line = sg.line;
    const float scale2 = p.scale2;

#pragma unroll 1
    for (int i = (stream - sh.stream_at(sg, 0)) & (streams - 1); i < n; i += streams) {
        const int key = (t0 + i) * kKeyTile + tr;
        const bool edge = (t0 + i + 1) * kKeyTile > lim0;     // some row does not see the whole tile
        // new token k sees the key if kv_len - q_len + k >= key: from this row on.
        // Past the last key no column sees it, the unused ones neither: what
        // lies there must not raise the other columns' references.
        const int seen = !edge ? 0 : (key >= sg.keys ? kRowTile
                                      : (key - sg.q.kv_len + sg.q.q_len - sg.tok) * p.plan.group - sg.head - coff);
        const uint32_t turn = sh.turn_at(sg, i);
        wait_bar(&M->b.s_full[turn][u], (st.phases >> turn) & 1u, ab);
        st.phases ^= 1u << turn;
        tc_fence_after();
        const uint32_t tS = tS0 + (turn ? kColS1 : 0u);
        float mul = scale2, lvs = 0.f, ivs = 1.f;
        if (F8) {
            const uint32_t at = line + (uint32_t)i;
            const int s = (int)(at % C::kScMod);
            wait_bar(&M->b.c_full[s], (at / C::kScMod) & 1u, ab);
            const uint8_t* sc = smem + C::kOffSc + s * C::kScBytes + tr * 4;
            mul *= *reinterpret_cast<const float*>(sc);
            float vs = *reinterpret_cast<const float*>(sc + C::kScBytes / 2);
            __syncwarp();
            // a wide tile's scales are read by two units
            if (lane == 0) mbar_arrive(&M->b.c_empty[s]);
            if (!wide && lane == 0) mbar_arrive(&M->b.c_empty[s]);
            if (edge && key >= sg.keys) vs = 1.f;             // no key here: any scale
            // Below 2^-100 (a row of zeros has scale 0) 1 / scale would take the sum
            // out of float32's range: there the sum counts the key with 2^-101, and
            // its weight for V is 0 (values below 2^-91 are dropped, not raised).
            if (vs < 3.944305e-31f) vs = 3.944305e-31f;
            lvs = lg2_approx(vs);
            ivs = ex2_approx(-lvs);
        }

        // base-2 exponents of the weights, relative to the references
        float t[32];
        const uint64_t mul2 = pack2(mul, mul), lvs2 = pack2(lvs, lvs);
#pragma unroll 1
        for (bool raised = false;; raised = true) {
            float top = -INFINITY;
            auto part = [&](auto first, auto count) {
                constexpr int c0 = decltype(first)::value, kB = decltype(count)::value;
                float x[kB];
                tmem_ldn<kB>(tS + (uint32_t)c0, x);
#pragma unroll
                for (int c = 0; c < kB; c += 2) {
                    uint64_t y = pack2(x[c], x[c + 1]);
                    const float2 r = *reinterpret_cast<const float2*>(&M->nref[u][c0 + c]);
                    if (F8) {
                        const float2 qm = *reinterpret_cast<const float2*>(&M->qm[u][c0 + c]);
                        y = fma2(mul2x(y, pack2(qm.x, qm.y)), mul2, add2(pack2(r.x, r.y), lvs2));
                    } else {
                        y = fma2(y, mul2, pack2(r.x, r.y));
                    }
                    unpack2(y, t[c0 + c], t[c0 + c + 1]);
                }
                if (edge) {
#pragma unroll
                    for (int c = 0; c < kB; ++c)
                        if (c0 + c < seen) t[c0 + c] = -INFINITY;
                }
#pragma unroll
                for (int c = 0; c < kB; ++c) top = fmaxf(top, t[c0 + c]);
            };
            part(std::integral_constant<int, 0>{}, std::integral_constant<int, (N < 16 ? N : 16)>{});
            if constexpr (N > 16) part(std::integral_constant<int, 16>{}, std::integral_constant<int, N - 16>{});
            // (raised once: scores of 2^28 and more round by more than the threshold)
            if (raised || !named_any(bar, 128, top > C::kLift + C::kLazy)) break;
            // one is too large: raise its reference to its largest score so far
#pragma unroll 1
            for (int c0 = 0; c0 < N; c0 += 4) {
                float x[4], mine = 0.f;
                tmem_ldn<4>(tS + (uint32_t)c0, x);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float y = fmaf(F8 ? x[c] * M->qm[u][c0 + c] : x[c], mul, lvs);
                    if (c0 + c < seen) y = -INFINITY;
                    y = redux_max(y);
                    if (lane == c) mine = y;
                }
                if (lane < 4) M->red[u][wq][c0 + lane] = mine;
            }
            named_sync(bar, 128);
            if (tr < N) {
                const float old = M->ref[u][tr];
                const float most = fmaxf(fmaxf(M->red[u][0][tr], M->red[u][1][tr]), fmaxf(M->red[u][2][tr], M->red[u][3][tr]));
                // each row by its own scores alone: the others' do not reach its bits
                const float ref = most > old + C::kLazy ? most : old;
                M->ref[u][tr] = ref;
                M->nref[u][tr] = C::kLift - ref;
                M->fac[u][tr] = ex2_approx(old - ref);
            }
            named_sync(bar, 128);
            if (lane < N) l *= M->fac[u][lane];
            if (i >= streams) {                            // the accumulator holds earlier tiles
                wait_bar(&M->b.pv_done[u], (st.tiles - 1u) & 1u, ab);
                tc_fence_after();
#pragma unroll 1
                for (int c0 = 0; c0 < N; c0 += 8) {
                    float o[8];
                    tmem_ldn<8>(tO + c0, o);
#pragma unroll
                    for (int c = 0; c < 8; ++c) o[c] *= M->fac[u][c0 + c];
                    tmem_st8(tO + c0, reinterpret_cast<const uint32_t(&)[8]>(o));
                }
                tmem_st_wait();
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M->b.s_free[turn][u]);
        // the P buffer is free once this unit's previous product is done
        if (st.tiles > 0) wait_bar(&M->b.pv_done[u], (st.tiles - 1u) & 1u, ab);
        ++st.tiles;
#pragma unroll
        for (int c0 = 0; c0 < N; c0 += 8) {
            uint32_t pk[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float& a = t[c0 + 2 * c];
                float& b = t[c0 + 2 * c + 1];
                a = ex2_approx(a);
                b = ex2_approx(b);
                // weights become 16-bit for the product with V (half a step: bf16
                // 2^-9, fp16 2^-12 of the binade); the sums keep them in float32
                if (F8) {
                    const __half2 h = __floats2half2_rn(a, b);
                    pk[c] = reinterpret_cast<const uint32_t&>(h);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                    pk[c] = reinterpret_cast<const uint32_t&>(h);
                }
            }
            *reinterpret_cast<uint4*>(P + (c0 / 8) * (kKeyTile * 16) + tr * 16) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        if (F8 && ivs > 1.2676506e30f) {                      // 2^100
#pragma unroll 1
            for (int c0 = 0; c0 < N; c0 += 8)
                *reinterpret_cast<uint4*>(P + (c0 / 8) * (kKeyTile * 16) + tr * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        if constexpr (F8) {
            // Widen V's e4m3 codes, 16 at a time; two units share a wide tile.
            // (The widened tile kW before this one has been multiplied, and so
            // has whatever the loaded tile's place held before.)
            const uint32_t at = line + (uint32_t)i;
            const int d = (int)(at % C::kW), s = (int)(at % C::kV);
            wait_bar(&M->b.w_empty[d], ((at / C::kW) & 1u) ^ 1u, ab);
            wait_bar(&M->b.v_full[s], (at / C::kV) & 1u, ab);
            const uint8_t* src = smem + C::kOffV + (size_t)s * C::kLoadBytes;
            uint8_t* dst = smem + C::kOffW + (size_t)d * C::kTileBytes;
            constexpr int kPieces = kKeyTile * HD / 16, kPer = HD / 16;
            const int valid = edge ? sg.keys - (t0 + i) * kKeyTile : kKeyTile;   // rows with a key
            // A thread's pieces lie `step` pieces, a multiple of 8 rows, apart: their
            // swizzle is the same.  It reads the two 8-byte halves of a piece in an
            // order that differs between lanes, so that neither the loads nor the
            // stores of a quarter warp meet in a bank.
            auto widen = [&](int x0, auto count, auto step) {
                constexpr int kN = decltype(count)::value, kStep = decltype(step)::value, kB = 2;
                const int row0 = x0 / kPer, c0 = (x0 % kPer) * 2, sw = row0 & 7;
                const int flip = HD == 128 ? ((tr >> 2) ^ (tr >> 3)) & 1 : (tr >> 3) & 1;
                const uint8_t* from = src + x0 * 16;
                uint8_t* to = dst + (c0 / 8) * C::kHalfBytes + row0 * 128;
                const int a = flip * 8, b = 8 - a;
                const int ta = (((c0 & 7) + flip) ^ sw) * 16, tb = (((c0 & 7) + 1 - flip) ^ sw) * 16;
#pragma unroll 1
                for (int h = 0; h < kN; h += kB) {
                    uint2 v[2 * kB];
#pragma unroll
                    for (int k = 0; k < kB; ++k) {
                        v[2 * k] = *reinterpret_cast<const uint2*>(from + k * kStep * 16 + a);
                        v[2 * k + 1] = *reinterpret_cast<const uint2*>(from + k * kStep * 16 + b);
                    }
#pragma unroll
                    for (int k = 0; k < kB; ++k) {
                        *reinterpret_cast<uint4*>(to + k * (kStep / kPer) * 128 + ta) = e4m3x8_to_half8(v[2 * k].x, v[2 * k].y);
                        *reinterpret_cast<uint4*>(to + k * (kStep / kPer) * 128 + tb) =
                            e4m3x8_to_half8(v[2 * k + 1].x, v[2 * k + 1].y);
                    }
                    from += kB * kStep * 16;
                    to += kB * (kStep / kPer) * 128;
                }
                // rows without a key become zeros, whatever their places hold
                if (valid < kKeyTile) {
#pragma unroll 1
                    for (int h = kN; h > 0; --h) {
                        to -= (kStep / kPer) * 128;
                        if (row0 + (h - 1) * (kStep / kPer) < valid) break;
                        *reinterpret_cast<uint4*>(to + ta) = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4*>(to + tb) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
            };
            if constexpr (wide)
                widen((u & 1) * 128 + tr, std::integral_constant<int, kPieces / 256>{}, std::integral_constant<int, 256>{});
            else
                widen(tr, std::integral_constant<int, kPieces / 128>{}, std::integral_constant<int, 128>{});
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M->b.p_full[u]);
        // the weights' sums (over w / scale for e4m3), while the product runs: a
        // row's sum in one lane, since a sum per row and thread would not fit
        // the registers
        if (F8) {
#pragma unroll
            for (int c = 0; c < N; ++c) t[c] *= ivs;
        }
        if constexpr (N == 24) {
            float* rest = t + 16;
            const float a = lane_sums<16>(t), b = lane_sums<8>(rest);
            l += lane < 16 ? a : b;
        } else {
            l += lane_sums<N>(t);
        }
    }

    // hand the sums on; the segment before the last has been read
    {
        M->red[u][wq][lane] = l;
        wait_bar(&M->b.e_free[parity], ((st.seg >> 1) & 1u) ^ 1u, ab);
        named_sync(bar, 128);
        if (tr < N) {
            M->fin_l[parity][u][tr] = (M->red[u][0][tr] + M->red[u][1][tr]) + (M->red[u][2][tr] + M->red[u][3][tr]);
            M->fin_m[parity][u][tr] = -M->nref[u][tr];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&M->b.l_done[parity]);
    }
    ++st.seg;
}

// The CTA of the last piece of an item that this CTA's span ends inside of.
__device__ __noinline__ int join_last(PlanInput p, int64_t total, int rest) {
    const int spans = plan_spans(p, total, (int)gridDim.x);
    return plan_owner(total, plan_cut(total, (int)blockIdx.x + 1, spans) + rest, spans);
}

// Joins the streams of a finished segment and stores it (128 threads).
template <int HD>
__device__ __forceinline__ void finish_segment(const PagedParams& p, const SegInfo& sg, Misc* M, uint32_t tmem,
                                               uint32_t seg) {
    volatile WaitState* ab = &M->wst;
    const Shape sh(sg.rows);
    const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int tr = wq * 32 + lane, parity = seg & 1;
    const int n = sg.n, used = min(n, sh.streams);            // streams with an accumulator
    const bool whole = n == sg.tiles;
    float* part = p.part + (size_t)(blockIdx.x * 2 + (sg.t0 == 0 ? 1 : 0)) * piece_floats(HD);
    int64_t at = -1;
    if (tr < sg.rows) {
        int i, g;
        plan_row(p.plan.group, sg.tok, sg.head, tr, i, g);
        at = (int64_t)(sg.q.a + i) * p.heads + (int64_t)sg.h * p.plan.group + g;
    }
    if (tr < kRowTile)
        M->row_at[tr] = at < 0 ? nullptr
                               : (whole ? reinterpret_cast<uint8_t*>(p.out + (size_t)at * HD)
                                        : reinterpret_cast<uint8_t*>(part + 2 * kRowTile + tr * HD));
    wait_bar(&M->b.l_done[parity], (seg >> 1) & 1u, ab);
    wait_bar(&M->b.o_done[parity], (seg >> 1) & 1u, ab);
    tc_fence_after();
    const bool store = !ab->abort;
    if (tr < sh.cols) {
        const int c = tr >= sh.width() ? tr - sh.width() : tr;
        // the unit that holds this column of the segment's k-th stream
        auto unit = [&](int k) {
            const int s = sh.stream_at(sg, k);
            return sh.wide ? 2 * s + (tr >= sh.width() ? 1 : 0) : s;
        };
        float m = kFloorRef;
#pragma unroll 1
        for (int k = 0; k < used; ++k) m = fmaxf(m, M->fin_m[parity][unit(k)][c]);
        float sum = 0.f;
#pragma unroll 1
        for (int k = 0; k < used; ++k) {
            sum = fmaf(M->fin_l[parity][unit(k)][c], ex2_approx(M->fin_m[parity][unit(k)][c] - m), sum);
        }
        const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
#pragma unroll 1
        for (int k = 0; k < used; ++k) M->join[unit(k)][c] = ex2_approx(M->fin_m[parity][unit(k)][c] - m) * inv;
        if (store && whole && p.lse && at >= 0) p.lse[at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
        if (store && !whole) {
            part[tr] = m;
            part[kRowTile + tr] = sum;
        }
    }
    if (tr == 0 && sg.t0 == 0 && !whole) p.desc[blockIdx.x] = JoinDesc{sg.r, sg.j, sg.h, join_last(p.plan, M->total, sg.rest)};
    named_sync(5, 128);
    const uint32_t tO = tmem + ((uint32_t)(wq * 32) << 16) + kColO * (1 + parity);
#pragma unroll 1
    for (int c0 = 0; c0 < sh.cols; c0 += 8) {
        float o[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] = 0.f;
#pragma unroll 1
        for (int k = 0; k < used; ++k) {
            float x[8];
            const int st = sh.stream_at(sg, k);
            const bool second = c0 >= sh.width();
            const float* f = &M->join[sh.wide ? 2 * st + second : st][second ? c0 - sh.width() : c0];
            tmem_ldn<8>(tO + sh.column(st) + (uint32_t)c0, x);
#pragma unroll
            for (int c = 0; c < 8; ++c) o[c] = fmaf(x[c], f[c], o[c]);
        }
        if (!store || tr >= HD) continue;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint8_t* row = M->row_at[c0 + c];
            if (!row) break;                                  // rows come first
            if (whole)
                reinterpret_cast<uint16_t*>(row)[tr] = __bfloat16_as_ushort(__float2bfloat16_rn(o[c]));
            else
                reinterpret_cast<float*>(row)[tr] = o[c];
        }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&M->b.e_free[parity]);
    named_sync(5, 128);                                       // row_at and join are no longer read
}

template <int HD, bool F8>
__global__ void __launch_bounds__(kThreads, 1)
    attn_paged_kernel(const __grid_constant__ Maps maps, const PagedParams p) {
    using C = Cfg<HD, F8>;
    extern __shared__ uint8_t smem_raw[];
    // an offset, not an address rounded as an integer: the compiler keeps to
    // shared-memory instructions
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    Misc* M = reinterpret_cast<Misc*>(smem + C::kOffMisc);
    // by a shuffle, so that the compiler knows it to be the same in every lane:
    // e4m3 blocks of 1 to 17 tokens 195 -> 184 us, e4m3 decoding 115.7 -> 113.5
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const PlanInput& pl = p.plan;
    const int cta = (int)blockIdx.x;
    pdl_launch_dependents();

    // ---------------- barriers and descriptors, beside the end of the kernel
    // before this one
    if (threadIdx.x < (int)(sizeof(Bars) / sizeof(uint64_t))) {
        mbar_init(reinterpret_cast<uint64_t*>(&M->b) + threadIdx.x, kBarCounts<F8>.n[threadIdx.x]);
        fence_mbar_init();
    } else if (threadIdx.x == 21 * 32) {
        M->wst.abort = 0;
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
    }
    pdl_wait();
    if (threadIdx.x == 22 * 32) M->wst.limit = ws_wait_limit(p.ws);
    if (threadIdx.x == 23 * 32) p.desc[cta] = JoinDesc{-1, 0, 0, 0};
    // ---------------- this CTA's span
    if (cta == 0) check_requests(pl.q_off, pl.kv_len, pl.R, pl.T, pl.most, p.ws);
    const int per = (pl.R + kThreads - 1) / kThreads;
    const int r0 = min((int)threadIdx.x * per, pl.R), r1 = min(r0 + per, pl.R);
    int64_t sum = 0;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) sum += plan_request_length(pl, r);
    int64_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) M->scan[warp] = upto;
    __syncthreads();
    const int64_t part = lane < kThreads / 32 ? M->scan[lane] : 0;
    int64_t parts = part;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, parts, o);
        if (lane >= o) parts += x;
    }
    const int64_t total = __shfl_sync(0xffffffffu, parts, 31);
    const int64_t base = upto - sum + __shfl_sync(0xffffffffu, parts - part, warp);
    const int spans = plan_spans(pl, total, (int)gridDim.x);
    if (cta >= spans) return;                                 // the same for every thread of the CTA
    const Span span = plan_span(total, cta, spans);
    const int64_t begin = span.begin, end = span.end;
    if (base <= begin && begin < base + sum) {
        int64_t at = base;
        int r = r0;
#pragma unroll 1
        for (; r < r1 - 1; ++r) {                             // it is the last one, if none before it
            const int64_t t = plan_request_length(pl, r);
            if (begin < at + t) break;
            at += t;
        }
        M->start_r = r;
        M->start_skip = begin - at;
    }
    if (threadIdx.x == 0) M->total = total;
    if (warp == 1) tmem_alloc(&M->tmem, kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = M->tmem;
    volatile WaitState* ab = &M->wst;
    // a role's next segment: false at the end or when a wait ran out
    uint32_t nseg = 0;
    SegInfo sg;
    auto next_segment = [&]() {
        const int at = nseg % kSegs;
        if (!__all_sync(0xffffffffu, wait_bar(&M->b.seg_full[at], (nseg / kSegs) & 1u, ab))) return false;
        sg = M->seg[at];
        return sg.rows > 0;
    };
    auto done_segment = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&M->b.seg_empty[nseg % kSegs]);
        ++nseg;
    };

    const int bp = min(1 << p.page_log2, kKeyTile);           // tokens of a page inside one tile
    const int ppt = kKeyTile / bp;                            // pages of a tile

    // ---------------- loads of K (warp 0) and V (warp 2) tiles
    // A place in the line of tiles: the next tile to load.
    struct Place {
        int tok, end, keys;                                   // first token of the tile, of the segment's end; keys
        int at, now, next;                                    // page table: lane's entries of 32 pages from `at`, and the 32 after
        int r, x;
        uint32_t seg, slot, phase, count;                     // segment; ring place; tiles issued
        uint64_t pol;
        bool more;
    };
    const int pg = lane & 7;
    const int lane_tok = pg < ppt ? pg * bp : 1 << 30;        // this lane's page of a tile, in tokens
    bool ok = true;
    auto entry = [&](const Place& c, int k) {
        return (int64_t)k << p.page_log2 < c.keys ? load4(p.page_table + (size_t)c.r * p.max_pages + k) : -1;
    };
    auto enter = [&](Place& c) {
        const int at = c.seg % kSegs;
        ok = ok && __all_sync(0xffffffffu, wait_bar(&M->b.seg_full[at], (c.seg / kSegs) & 1u, ab));
        const SegInfo& s = M->seg[at];
        c.more = ok && s.rows > 0;
        if (!c.more) return;
        c.tok = s.t0 * kKeyTile;
        c.end = (s.t0 + s.n) * kKeyTile;
        c.keys = s.keys;
        c.r = s.r;
        c.x = s.h << p.page_log2;
        // more than one row tile of a request reads its keys again
        c.pol = (int64_t)s.q.q_len * pl.group > kRowTile ? policy_evict_normal() : policy_evict_first();
        c.at = (c.tok >> p.page_log2) & ~31;
        c.now = entry(c, c.at + lane);
        c.next = entry(c, c.at + 32 + lane);
    };
    // this lane's page of the place's tile (pages past the keys: any)
    auto page_of = [&](Place& c) {
        int rel = (c.tok >> p.page_log2) - c.at;
        if (rel >= 32) {
            rel -= 32;
            c.at += 32;
            c.now = c.next;
            c.next = entry(c, c.at + 32 + lane);
        }
        return __shfl_sync(0xffffffffu, c.now, (rel + pg) & 31);
    };
    // on to the next tile; true if it is another segment's
    auto step = [&](Place& c) {
        ++c.count;
        c.tok += kKeyTile;
        if (c.tok < c.end) return false;
        ++c.seg;
        return true;
    };
    auto load = [&](auto which, Place& c, int id) {
        constexpr bool kIsV = decltype(which)::value;
        constexpr uint32_t kRing = kIsV ? C::kV : C::kK;
        uint64_t* full = (kIsV ? M->b.v_full : M->b.k_full) + c.slot;
        ok = ok && __all_sync(0xffffffffu, wait_bar((kIsV ? M->b.v_empty : M->b.k_empty) + c.slot, c.phase ^ 1u, ab));
        const uint32_t cs = c.count % C::kScMod;
        if (F8 && !kIsV)
            ok = ok && __all_sync(0xffffffffu, wait_bar(&M->b.c_empty[cs], ((c.count / C::kScMod) & 1u) ^ 1u, ab));
        if (!ok) return;
        const bool valid = lane_tok < c.keys - c.tok;
        if (valid && (uint32_t)id >= (uint32_t)p.n_pages) {
            raise_status(p.ws, kStatBadPage);
            id = p.n_pages;                                   // past the tensor: zeros
        }
        const uint32_t pages = __popc(__ballot_sync(0xffffffffu, valid) & 0xFFu);
        const int x = c.x + (ppt == 1 ? c.tok & ((1 << p.page_log2) - 1) : 0);        // a 256-token page is two tiles
        if (elect_one()) {
            mbar_expect_tx(full, pages * (uint32_t)(bp * (F8 ? HD : HD * 2)));
        }
        __syncwarp();
        uint8_t* dst = smem + (kIsV ? C::kOffV : 0) + c.slot * C::kLoadBytes;
        if (F8 && !kIsV) {
            // the tile's 2 x 128 scales, 4 tokens to a lane: a tensor copy per page,
            // 64 bytes each at 16 tokens, took 248 us where this took 216 (64
            // requests of 8192 tokens, 8 heads of 128; 208 by now)
            const int tk = lane * 4;
            const uint32_t pid = (uint32_t)__shfl_sync(0xffffffffu, id, tk >> (p.page_log2 < 7 ? p.page_log2 : 7));
            const bool in = tk < c.keys - c.tok && pid < (uint32_t)p.n_pages;
            const size_t at = in ? (((size_t)pid * pl.kv_heads) << p.page_log2) + x + (tk & (bp - 1)) : 0;
            uint8_t* sc = smem + C::kOffSc + cs * C::kScBytes + lane * 16;
            cp_async16_zf(sc, p.k_scale + at, in ? 16u : 0u);
            cp_async16_zf(sc + C::kScBytes / 2, p.v_scale + at, in ? 16u : 0u);
            cp_async_arrive(&M->b.c_full[cs]);
        }
#pragma unroll 1
        for (uint32_t k = 0; k < pages; ++k) {
            const int pid = __shfl_sync(0xffffffffu, id, k);
            if (elect_one()) {
#pragma unroll
                for (int hf = 0; hf < (F8 ? 1 : C::kHalves); ++hf)
                    tma_load_3d(dst + hf * C::kHalfBytes, kIsV ? &maps.v : &maps.k, full, hf * 64, x, pid, c.pol);
            }
            dst += bp * (F8 ? HD : 128);
        }
        __syncwarp();
        if (++c.slot == kRing) {
            c.slot = 0;
            c.phase ^= 1u;
        }
    };
    // copies in flight of a ring, after an abort
    auto drain = [&](uint64_t* full, uint32_t ring, uint32_t count) {
        if (ab->abort && lane == 0)
#pragma unroll 1
            for (uint32_t k = count > ring ? count - ring : 0; k < count; ++k)
                mbar_wait_for(&full[k % ring], (k / ring) & 1u, ab->limit);
        __syncwarp();
    };

    if (warp == 0) {
        // ---------------- K tiles
        Place c = {};
        enter(c);
#pragma unroll 1
        while (ok && c.more) {
            load(std::false_type{}, c, page_of(c));
            if (!ok) break;
            const uint32_t seg = c.seg;
            if (step(c)) {
                if (lane == 0) mbar_arrive(&M->b.seg_empty[seg % kSegs]);
                enter(c);
            }
        }
        drain(M->b.k_full, C::kK, c.count);
        if (F8) drain(M->b.c_full, C::kScMod, c.count);
    } else if (warp == 1) {
        // ---------------- scores S^T = K Q^T
        // A stream's columns are free once the weights of its tile before are
        // made; at a change of shape, once all earlier weights are.
        const uint64_t dk = F8 ? desc_f8<HD>(smem) : smem_desc_sw128(smem, 16, 1024);
        const uint64_t dq = F8 ? desc_f8<HD>(smem + C::kOffQ) : smem_desc_sw128(smem + C::kOffQ, 16, 1024);
        uint32_t ks = 0, kph = 0;
        uint32_t free_ph = 0xFFu;      // by score tile (turn, unit): parity of its next s_free
        uint32_t run = 0, runs = 0;
        auto wait = [&](uint64_t* bar, uint32_t par) { ok = ok && __all_sync(0xffffffffu, wait_bar(bar, par, ab)); };
        auto give = [&](int u, uint32_t turn) {
            wait(&M->b.s_free[turn][u], (free_ph >> (4 * turn + u)) & 1u);
            free_ph ^= 1u << (4 * turn + u);
        };
#pragma unroll 1
        for (; ok && next_segment(); done_segment()) {
            const Shape sh(sg.rows);
            const uint32_t id = F8 ? idesc_e4m3_f32(128, sh.cols) : idesc_bf16_f32(128, sh.cols, false, false);
            const uint64_t b = dq + (sg.qp == 1 ? C::kQBytes / 16 : 0);
            // rows between Q's halves along head_dim (bf16), or between hi and lo
            const int q_rows = sg.qp == 2 ? 2 * C::kQRows : C::kQRows;
            if (sg.run != run) {
                // columns and buffers change hands: all products so far are done
                wait(&M->b.r_done, runs++ & 1u);
                run = sg.run;
            }
            q_places(sg, [&](int k, uint32_t use) { wait(&M->b.q_full[k], use & 1u); });
#pragma unroll 1
            for (int i = 0; ok && i < sg.n; ++i) {
                const int st = sh.stream_at(sg, i);
                const int u0 = sh.wide ? 2 * st : st;
                const uint32_t turn = sh.turn_at(sg, i);
                give(u0, turn);
                if (sh.wide) give(u0 + 1, turn);
                wait(&M->b.k_full[ks], kph);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t d = tmem + sh.column(st) + (turn ? kColS1 : 0u);
                    const uint64_t a = dk + ks * (C::kLoadBytes / 16);
                    if (F8) {
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk)   // hi, then lo
                            umma_f8(d, a + (kk % (HD / 32)) * 2, b + (uint32_t)((kk / (HD / 32)) * (q_rows * HD / 16) + (kk % (HD / 32)) * 2),
                                    id, kk ? 1u : 0u);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk)
                            umma_bf16(d, a + (kk / 4) * (C::kHalfBytes / 16) + (kk % 4) * 2,
                                      b + (uint32_t)((kk / 4) * (q_rows * 8) + (kk % 4) * 2), id, kk ? 1u : 0u);
                    }
                    umma_commit(&M->b.s_full[turn][u0]);
                    if (sh.wide) umma_commit(&M->b.s_full[turn][u0 + 1]);
                    umma_commit(&M->b.k_empty[ks]);
                    if (i == sg.n - 1) q_places(sg, [&](int k, uint32_t) { umma_commit(&M->b.q_empty[k]); });
                }
                __syncwarp();
                if (++ks == C::kK) {
                    ks = 0;
                    kph ^= 1u;
                }
            }
        }
        if (elect_one()) umma_commit(&M->b.done);
        __syncwarp();
    } else if (warp == 3) {
        // ---------------- products O^T += V^T P^T
        constexpr uint32_t a_lbo = HD == 128 ? C::kHalfBytes : 0;   // head_dim 64: rows 64..127 repeat 0..63
        const uint64_t dv = smem_desc_sw128(smem + (F8 ? C::kOffW : C::kOffV), a_lbo, 1024);
        const uint64_t dp = smem_desc_plain(smem + C::kOffP, 128, kKeyTile * 16);
        uint32_t vs = 0, vph = 0, ws = 0, run = 0;
        uint32_t made = 0;                                    // parity of each unit's next p_full, by bit
        auto wait = [&](uint64_t* bar, uint32_t par) { ok = ok && __all_sync(0xffffffffu, wait_bar(bar, par, ab)); };
#pragma unroll 1
        for (; ok && next_segment(); done_segment()) {
            const Shape sh(sg.rows);
            const uint32_t id = F8 ? idesc_f16_f32(128, sh.cols, true, true) : idesc_bf16_f32(128, sh.cols, true, true);
            const uint32_t set = tmem + kColO * (1u + (nseg & 1u));
            if (sg.run != run && elect_one()) umma_commit(&M->b.r_done);
            __syncwarp();
            run = sg.run;
#pragma unroll 1
            for (int i = 0; ok && i < sg.n; ++i) {
                const int st = sh.stream_at(sg, i), u0 = sh.wide ? 2 * st : st;
                // bf16: the V tile as it was loaded; e4m3: the widened one, which
                // p_full covers, as it does the end of the reads of the loaded one
                if (!F8) {
                    wait(&M->b.v_full[vs], vph);
                    const int valid = sg.keys - (sg.t0 + i) * kKeyTile;
                    if (ok && valid < kKeyTile) {
                        // rows past the last key hold whatever the pages or this buffer held
                        uint8_t* vt = smem + C::kOffV + (size_t)vs * C::kTileBytes;
#pragma unroll 1
                        for (int k = max(valid, 0) * 8 + lane; k < kKeyTile * 8; k += 32)
#pragma unroll
                            for (int hf = 0; hf < C::kHalves; ++hf)
                                *reinterpret_cast<uint4*>(vt + hf * C::kHalfBytes + k * 16) = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async();
                        __syncwarp();
                    }
                }
                wait(&M->b.p_full[u0], (made >> u0) & 1u);
                if (sh.wide) wait(&M->b.p_full[u0 + 1], (made >> (u0 + 1)) & 1u);
                made ^= (sh.wide ? 3u : 1u) << u0;
                if (i == 0) wait(&M->b.e_free[nseg & 1], ((nseg >> 1) & 1u) ^ 1u);   // this set's last segment is stored
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t a = dv + (F8 ? ws : vs) * (C::kTileBytes / 16), b = dp + u0 * (C::kPBytes / 16);
                    const uint32_t d = set + sh.column(st);
                    umma_bf16(d, a, b, id, i >= sh.streams ? 1u : 0u);
#pragma unroll
                    for (int kk = 1; kk < kKeyTile / 16; ++kk) umma_bf16(d, a + kk * 128, b + kk * 16, id, 1u);
                    if (F8) mbar_arrive(&M->b.v_empty[vs]);
                    umma_commit(F8 ? &M->b.w_empty[ws] : &M->b.v_empty[vs]);
                    umma_commit(&M->b.pv_done[u0]);
                    if (sh.wide) umma_commit(&M->b.pv_done[u0 + 1]);
                    if (i == sg.n - 1) umma_commit(&M->b.o_done[nseg & 1]);
                }
                __syncwarp();
                if (++vs == C::kV) {
                    vs = 0;
                    vph ^= 1u;
                }
                if (F8 && ++ws == C::kW) ws = 0;
            }
        }
        // the tensor core is idle before its memory is given back
        if (elect_one()) {
            umma_commit(&M->b.done);
            mbar_wait_for(&M->b.done, 0, ab->limit);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---------------- segments and V tiles
        Cursor cur;
        cur.start(pl, M->start_r, M->start_skip, end - begin);
        uint32_t made = 0, line = 0, run = 0;                 // segments listed, their key tiles
        bool wide = false, more = true;
        int place = 0;                                        // the next Q place
        uint32_t use = 0;
        Place c = {};
        for (;;) {
            // before each segment's tiles, list it and those after it that there is
            // room for (the others never need more to get through this one)
#pragma unroll 1
            while (more) {
                uint64_t* bar = &M->b.seg_empty[made % kSegs];
                const uint32_t par = ((made / kSegs) & 1u) ^ 1u;
                if (made == c.seg)
                    ok = __all_sync(0xffffffffu, wait_bar(bar, par, ab));
                else if (!__all_sync(0xffffffffu, mbar_test(bar, par)))
                    break;
                if (!ok) break;
                Segment s;
                more = cur.next(pl, s);
                if (more && Shape(s.rows).wide != wide) {
                    wide = !wide;
                    run = line;
                }
                const bool both = more && Shape(s.rows).cols > C::kQRows;
                if (lane == 0) {
                    SegInfo& o = M->seg[made % kSegs];
                    o.rows = 0;
                    if (more)
                        o = SegInfo{s.r, s.j, s.h, s.t0, s.t1 - s.t0, s.tiles, s.keys, s.rows, s.tok, s.head, s.rest, line, run,
                                    both ? 2 : place, use, s.q};
                    mbar_arrive(&M->b.seg_full[made % kSegs]);
                }
                __syncwarp();
                if (more) line += (uint32_t)(s.t1 - s.t0);
                use += (both || place == 0 ? 1u : 0u) + (both || place == 1 ? 0x10000u : 0u);
                use &= 0x7FFF7FFFu;                           // parities are what counts
                if (!both) place ^= 1;
                ++made;
            }
            if (!ok) break;
            enter(c);
            if (!c.more) break;
            bool last = false;
#pragma unroll 1
            while (ok && !last) {
                load(std::true_type{}, c, page_of(c));
                last = step(c);
            }
            if (!ok) break;
            if (lane == 0) mbar_arrive(&M->b.seg_empty[(c.seg - 1) % kSegs]);
        }
        drain(M->b.v_full, C::kV, c.count);
    } else if (warp >= 4 + 4 * kUnits) {
        // ---------------- Q rows of the segment to come, and the finished one
        constexpr int kLanes = HD / 8, kStep = 128 / kLanes;  // 8 values per lane; rows per step
        const int ft = threadIdx.x - 32 * (4 + 4 * kUnits);
        // segment k's rows into its Q buffer; false at the end or when a wait ran out
        auto bring = [&](uint32_t k) {
            const SegInfo& s = M->seg[k % kSegs];
            bool got = wait_bar(&M->b.seg_full[k % kSegs], (k / kSegs) & 1u, ab);
            if (got && s.rows > 0)
                q_places(s, [&](int b, uint32_t use) { got = got && wait_bar(&M->b.q_empty[b], (use & 1u) ^ 1u, ab); });
            if (named_any(5, 128, !got)) return false;
            if (s.rows == 0) return false;
            const int cols = Shape(s.rows).cols, q_rows = s.qp == 2 ? 2 * C::kQRows : C::kQRows;
            uint8_t* qt = smem + C::kOffQ + (s.qp == 1 ? C::kQBytes : 0);
            const int x = ft % kLanes;
#pragma unroll 1
            for (int row = ft / kLanes; row < cols; row += kStep) {
                int i, gq;
                plan_row(pl.group, s.tok, s.head, row, i, gq);
                const bool in = row < s.rows;
                const uint16_t* src = in ? p.q + (int64_t)(s.q.a + i) * p.q_stride + ((int64_t)s.h * pl.group + gq) * HD + x * 8
                                         : p.q;
                if (!F8) {
                    cp_async16_zf(qt + (x / 8) * (q_rows * 128) + row * 128 + ((x ^ row) & 7) * 16, src, in ? 16u : 0u);
                } else {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (in) v = load16(src);
                    uint2 hi, lo;
                    const float sc = split_e4m3<kLanes>(v, hi, lo);
                    *reinterpret_cast<uint2*>(qt + swz_f8<HD>(row, x / 2) + (x & 1) * 8) = hi;
                    *reinterpret_cast<uint2*>(qt + swz_f8<HD>(q_rows + row, x / 2) + (x & 1) * 8) = lo;
                    if (x == 0) M->q_scale[(s.qp == 1 ? C::kQRows : 0) + row] = sc;
                }
            }
            if (!F8) cp_async_wait_all();
            fence_proxy_async();
            q_places(s, [&](int b, uint32_t) { mbar_arrive(&M->b.q_full[b]); });
            return true;
        };
        bool have = bring(0), after = have && bring(1);
#pragma unroll 1
        for (; have; ++nseg) {
            finish_segment<HD>(p, M->seg[nseg % kSegs], M, tmem, nseg);
            if (lane == 0) mbar_arrive(&M->b.seg_empty[nseg % kSegs]);
            have = after;
            after = after && bring(nseg + 2);
        }
    } else {
        // ---------------- softmax
        const int u = (warp - 4) >> 2;
        SoftState st = {0, 0, 0};
#pragma unroll 1
        for (;; ++nseg) {
            const int at = nseg % kSegs;
            const bool got = wait_bar(&M->b.seg_full[at], (nseg / kSegs) & 1u, ab);
            // the unit agrees on whether there is a segment; what the one before
            // left in its shared memory is no longer read
            if (named_any(1 + u, 128, !got)) break;
            const SegInfo& s = M->seg[at];
            if (s.rows == 0) break;
            // a loop for each number of rows: without the one for 48, e4m3 blocks of 1
            // to 17 tokens take 229 us where they take 180, and 48 rows over long e4m3
            // caches 146 and 138; without the one for 8, e4m3 decoding 115.4 and 113.5.
            // (bf16 has no loop for 24: such items are bound by the cache's bytes, and
            // one shape more cost blocks of 1 to 17 tokens 4 %.)
            if (s.rows <= 8)
                soft_segment<HD, F8, 8>(p, s, M, smem, tmem, u, st);
            else if (s.rows <= 16)
                soft_segment<HD, F8, 16>(p, s, M, smem, tmem, u, st);
            else if (F8 && s.rows <= 24)
                soft_segment<HD, F8, F8 ? 24 : 32>(p, s, M, smem, tmem, u, st);
            else if (s.rows <= 32)
                soft_segment<HD, F8, 32>(p, s, M, smem, tmem, u, st);
            else if (s.rows <= 48)
                soft_segment<HD, F8, 48>(p, s, M, smem, tmem, u, st);
            else
                soft_segment<HD, F8, 64>(p, s, M, smem, tmem, u, st);
            __syncwarp();
            if (lane == 0) mbar_arrive(&M->b.seg_empty[at]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && M->wst.abort) raise_status(p.ws, kStatTimeout);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

// ------------------------------------------------------------------ join
// out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i over an item's pieces,
// m their largest reference.  Latency only: at most two pieces per CTA, 10 MB
// of them; launched beside the kernel above, it adds about 3 us.
// Block (c, y) joins 8 rows of the item that starts in CTA c's span and ends
// in a later one: a warp per row, pieces in the order of the keys.
template <int HD>
__global__ void __launch_bounds__(256) attn_paged_join(const PagedParams p, int grid) {
    pdl_launch_dependents();
    pdl_wait();
    const JoinDesc d = p.desc[blockIdx.x];
    const int c = blockIdx.x, row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (d.r < 0 || d.last >= grid) return;
    const PlanInput& pl = p.plan;
    const Request q = plan_request(pl, d.r);
    const int64_t rho = (int64_t)d.j * kRowTile + row;
    if (rho >= (int64_t)q.q_len * pl.group) return;
    auto piece = [&](int i) { return p.part + (size_t)(i == c ? 2 * c + 1 : 2 * i) * piece_floats(HD); };
    float m = kFloorRef;
#pragma unroll 1
    for (int i = c + lane; i <= d.last; i += 32) m = fmaxf(m, piece(i)[row]);
    m = warp_max(m);
    constexpr int N = HD / 32;
    float o[N], l = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int i = c; i <= d.last; ++i) {
        const float* x = piece(i);
        const float f = ex2_approx(x[row] - m);
        l = fmaf(x[kRowTile + row], f, l);
        const float* v = x + 2 * kRowTile + row * HD + lane;
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = fmaf(v[e * 32], f, o[e]);
    }
    const int i = (int)(rho / pl.group), g = (int)(rho - (int64_t)i * pl.group);
    const int64_t at = (int64_t)(q.a + i) * p.heads + (int64_t)d.h * pl.group + g;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < N; ++e)
        p.out[(size_t)at * HD + e * 32 + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(o[e] * inv));
    if (p.lse && lane == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// PlanInput::lengths.  The lengths stand for the time a CTA takes, fitted to
// mixed batches of both head sizes, by the rows and the cache's type alone (an
// item costs about what two tiles do, between its Q rows and its stored rows;
// e4m3 tiles of many rows cost more than they bring in bytes).  With every tile
// as long as another, blocks of 1 to 17 tokens (64 requests of 1000 to 6001
// keys, 48 heads of 64) take 196 us where they take 180 over e4m3 caches, and 127
// and 120 over bf16; blocks of 1 to 6 tokens (256 requests of 200 to 4000, or of
// 50 to 1000 keys) take the same.
constexpr uint32_t tile_lengths(uint32_t r8, uint32_t r16, uint32_t r24, uint32_t r32, uint32_t r48, uint32_t r64) {
    return r8 | r16 << 5 | r24 << 10 | r32 << 15 | r48 << 20 | r64 << 25;
}

template <int HD, bool F8>
cudaError_t launch(const Maps& maps, const PagedParams& p, int grid, cudaStream_t s) {
    const size_t smem = smem_bytes<HD, F8>();
    cudaError_t e = allow_smem(attn_paged_kernel<HD, F8>, smem);
    if (e != cudaSuccess) return e;
    prof_begin(kPAttnPaged, s);
    e = launch_kernel(attn_paged_kernel<HD, F8>, dim3(grid), dim3(kThreads), smem, s, true, maps, p);
    prof_end(s);
    if (e != cudaSuccess) return e;
    prof_begin(kPAttnPagedJoin, s);
    e = launch_kernel(attn_paged_join<HD>, dim3(grid, kRowTile / 8), dim3(256), 0, s, true, p, grid);
    prof_end(s);
    return e;
}

}  // namespace

size_t attn_paged_workspace_bytes(int, int, int, int, int head_dim) {
    const size_t grid = (size_t)num_sms();
    return sizeof(WsHeader) + align_up(grid * sizeof(JoinDesc), 256) +
           grid * 2 * (size_t)kRowTile * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_attn_paged(const void* q, int64_t q_stride, const dspark_kv_cache_t& c, const dspark_kv_batch_t& b,
                              int n_heads, float scale, void* out, float* lse, void* ws, cudaStream_t s) {
    const int grid = num_sms();
    uint8_t* w = static_cast<uint8_t*>(ws) + sizeof(WsHeader);
    PagedParams p;
    const bool f8 = c.dtype == DSPARK_E4M3;
    p.q = static_cast<const uint16_t*>(q);
    p.q_stride = q_stride;
    // with no more items than CTAs every CTA has about one piece, whatever item
    // it is of, and short spans let more CTAs in (one request of 777 keys, 8
    // heads: 13.2 us on the device against 14.0)
    const bool few = (b.R + (int64_t)b.T * (n_heads / c.n_kv_heads) / kRowTile) * c.n_kv_heads <= grid;
    p.plan = PlanInput{b.q_off, b.kv_len, b.R, b.T, n_heads / c.n_kv_heads, c.n_kv_heads, (int64_t)b.max_pages * c.page,
                       few ? 0 : (f8 ? 12 : 8), f8 ? tile_lengths(4, 4, 4, 5, 6, 7) : tile_lengths(4, 4, 4, 4, 5, 6)};
    p.page_table = b.page_table;
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.ws = ws;
    p.desc = reinterpret_cast<JoinDesc*>(w);
    p.part = reinterpret_cast<float*>(w + align_up((size_t)grid * sizeof(JoinDesc), 256));
    p.max_pages = b.max_pages;
    p.n_pages = c.n_pages;
    p.page_log2 = ceil_log2_i(c.page);
    p.heads = n_heads;
    p.scale2 = scale * kLog2e;
    // a page's planes of all heads are one run of n_kv_heads * page rows; the
    // page is a dimension of its own, so coordinates stay small and an id past
    // the last page reads zeros
    Maps maps;
    const cuuint64_t hd = (cuuint64_t)c.head_dim, rows = (cuuint64_t)c.n_kv_heads * c.page, pages = (cuuint64_t)c.n_pages;
    const cuuint32_t bp = (cuuint32_t)(c.page < kKeyTile ? c.page : kKeyTile);
    const cuuint64_t es = f8 ? 1 : 2;
    const cuuint64_t dims[3] = {hd, rows, pages}, str[2] = {hd * es, rows * hd * es};
    const cuuint32_t box[3] = {f8 ? (cuuint32_t)hd : 64u, bp, 1};
    const CUtensorMapDataType dt = f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    // e4m3: K feeds the tensor core in rows of head_dim bytes, V the widening
    const CUtensorMapSwizzle swz_k = f8 && hd == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    const CUtensorMapSwizzle swz_v = f8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
    const bool ok = make_tensor_map(&maps.k, dt, 3, c.k, dims, str, box, swz_k) &&
              make_tensor_map(&maps.v, dt, 3, c.v, dims, str, box, swz_v);
    if (!ok) return cudaErrorInvalidValue;
    if (c.head_dim == 64) return f8 ? launch<64, true>(maps, p, grid, s) : launch<64, false>(maps, p, grid, s);
    return f8 ? launch<128, true>(maps, p, grid, s) : launch<128, false>(maps, p, grid, s);
}

}  // namespace dspark
