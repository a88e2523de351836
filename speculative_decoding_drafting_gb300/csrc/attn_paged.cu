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
//
// One persistent CTA per SM walks an equal span of the line of all items' key
// tiles (attn_plan.h); pieces of split items go to the workspace and a second
// launch joins them in a fixed order.
//
//   warp 0      TMA producer: K and V tiles page by page (a page id out of
//               range lies past the tensor's end, so it reads as zeros)
//   warp 1      MMA issuer
//   warp 2      Q rows of the next item (e4m3 caches: split, see below)
//   warp 3      the list of this CTA's segments, a few ahead of the others
//   warps 4-19  four softmax units of four warps, 32 rows of Q each.  Items of
//               up to 32 rows go through four streams of key tiles (unit u
//               takes every fourth), wider ones through two streams of two
//               units, each stream with its own references, sums and
//               accumulator, so that some exponentiate while the products of
//               others run.  Thread = key, registers = rows.  The reference of
//               a row is raised only when a score exceeds it by more than 2^8
//               (a vote per tile; p <= 2^8 is far inside bf16 and float32), so
//               a tile costs no maximum over its keys.
//
// e4m3 caches: K tiles go to the tensor core as they are.  Each row of Q is
// split into 2^e (hi + lo / 16) with hi, lo in e4m3, 2^e such that the row's
// largest value is in [128, 256): bf16's 8 significant bits are two times
// e4m3's 4, so the split is exact down to 2^-22 of the row's largest value.
// hi and lo are 2 x N columns of one product of twice bf16's rate.  V is
// widened to bf16 instead, since weights want more than a few terms of 4 bits;
// the units that made a tile's weights do it, the one shared-memory pass that
// e4m3 costs.
//
// Keys a row must not see get weight 0 by selection, not by multiplication;
// V rows past the item's last key are zeroed in shared memory, since 0 times
// a stale NaN would be NaN (widened e4m3 codes are always finite).
#include <type_traits>

#include <cuda.h>

#include "attn_plan.h"
#include "kernels.h"
#include "kv.cuh"
#include "profile.h"
#include "sm100.cuh"

namespace dspark {

namespace {

constexpr float kFloorRef = -1e30f;     // reference before any score: finite, below every score
constexpr float kLazy = 8.f;            // bits a score may exceed its reference by

constexpr int kUnits = 4;               // softmax units of 128 threads
constexpr int kUnitRows = 32;           // columns of S^T a unit handles

template <int HD, bool F8>
struct Cfg {
    static constexpr int kTileBytes = kKeyTile * HD * 2;                   // a K or V tile as bf16
    static constexpr int kHalves = HD / 64;                                // 128-byte swizzle atoms of a row
    static constexpr int kHalfBytes = kKeyTile * 128;
    static constexpr int kLoadBytes = F8 ? kKeyTile * HD : kTileBytes;     // a tile as it lies in the cache
    static constexpr int kK = F8 ? (HD == 128 ? 3 : 6) : (HD == 128 ? 2 : 5);       // K tiles on the way
    static constexpr int kV = F8 ? (HD == 128 ? 2 : 4) : (HD == 128 ? 3 : 5);       // V tiles
    static constexpr int kW = F8 ? 2 : 0;                                  // widened V tiles
    static constexpr int kSc = F8 ? 4 : 0;                                 // scales of a tile (K, V)
    static constexpr int kScBytes = 2048;                                  // 2 x 128 scales, 16-token pages at 128-byte pitch
    static constexpr int kPBytes = kKeyTile * kUnitRows * 2;               // a unit's P^T
    static constexpr int kQBytes = kRowTile * HD * 2;                      // bf16 rows, or hi and lo
    static constexpr int kQ = F8 ? 2 : 1;
    static constexpr int kWMod = kW ? kW : 1, kScMod = kSc ? kSc : 1;      // divisors (unused without e4m3)
    static constexpr uint32_t kColO = F8 ? 256 : 128;                      // TMEM column of the accumulators
    static constexpr uint32_t kTmem = F8 ? 512 : 256;
    static constexpr int kOffV = kK * kLoadBytes;
    static constexpr int kOffW = kOffV + kV * kLoadBytes;
    static constexpr int kOffP = kOffW + kW * kTileBytes;
    static constexpr int kOffQ = kOffP + kUnits * kPBytes;
    static constexpr int kOffSc = kOffQ + kQ * kQBytes;
    static constexpr int kOffMisc = kOffSc + kSc * kScBytes;
};
constexpr int kThreads = 32 * (4 + 4 * kUnits);
constexpr uint32_t kReaders = 3 + 4 * kUnits;                              // warps that read a segment
constexpr int kSegs = 4;                // segments in flight between the roles

// A segment as the roles read it from shared memory (rows = 0: the end).
struct SegInfo {
    int r, j, h;
    int t0, n, tiles;                  // key tiles [t0, t0 + n) of tiles
    int keys, rows;
    Request q;
};

struct alignas(16) Misc {
    SegInfo seg[kSegs];
    uint64_t seg_full[kSegs], seg_empty[kSegs];
    float nref[kUnits][kUnitRows];     // minus the reference of a row
    float qm[kUnits][kUnitRows];       // 2^e of a row's split
    float fac[kUnits][kUnitRows];      // factor of a raised reference, then of the join
    float red[kUnits][4][kUnitRows];   // per-warp maxima, then sums
    int lim[kUnits][kUnitRows];        // keys a row sees
    float q_scale[2][kRowTile];        // 2^e of the Q buffers' rows
    int64_t row_at[2][kRowTile];       // a row's place in out's rows (-1: no row), by parity of the segment
    int64_t scan[32];
    int64_t total, start_skip;
    int start_r;
    uint32_t tmem;
    WaitState wst;
    uint64_t k_full[6], k_empty[6], v_full[5], v_empty[5];
    uint64_t w_empty[2];               // widened V tiles (p_full says that one is made)
    uint64_t c_full[4], c_empty[4];    // scales
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[kUnits], p_full[kUnits], pv_done[kUnits];
    uint64_t o_free, done;
};

template <int HD, bool F8>
constexpr size_t smem_bytes() {
    return 1024 + Cfg<HD, F8>::kOffMisc + sizeof(Misc);
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
    CUtensorMap k, v, ks, vs;
};

// Sums over the 32 lanes of N = 16 or 32 values per lane; lane i gets the sum
// of value i % N.
template <int N>
__device__ __forceinline__ float lane_sums(float (&x)[N]) {
    const int lane = threadIdx.x & 31;
    if constexpr (N == 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], 16);
    }
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = up ? x[i + o] : x[i], give = up ? x[i] : x[i + o];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    return x[0];
}

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

// One lane's 8 values of a Q row that `LANES` lanes share: e4m3 codes of hi
// and lo with q = 2^e (hi + lo / 16), and 2^e (NaN for a row that is not
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
        l[i] = __nv_cvt_float2_to_fp8x2(make_float2((a - f.x) * 16.f, (b - f.y) * 16.f), __NV_SATFINITE, __NV_E4M3);
    }
    hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
    return big >= 0x7F80u ? NAN : scale;
}

// A row tile's layout over units: width (columns of Q in use), streams.
struct Shape {
    int cols, streams;
    bool wide;
    __device__ __forceinline__ explicit Shape(int rows)
        : cols(rows <= 16 ? 16 : (rows <= 32 ? 32 : 64)), streams(rows > 32 ? 2 : 4), wide(rows > 32) {}
    __device__ __forceinline__ int stream_of(int unit) const { return wide ? unit >> 1 : unit; }
    // TMEM columns of a stream's scores (e4m3: lo follows hi after cols columns)
    template <bool F8>
    __device__ __forceinline__ uint32_t scores(int stream) const {
        return (uint32_t)stream * (F8 ? (wide ? 128u : 64u) : (wide ? 64u : 32u));
    }
    __device__ __forceinline__ uint32_t accum(int stream) const { return (uint32_t)stream * (wide ? 64u : 32u); }
};

// ------------------------------------------------------------------ softmax
struct SoftState {
    uint32_t tiles;                    // key tiles this unit has taken
    uint32_t line;                     // key tiles of all streams so far
    uint32_t seg;                      // segments so far
};

// Output columns [c0, c0 + K) of the item: the streams' accumulators times
// their factors.
template <int HD, int K>
__device__ __forceinline__ void store_columns(const PagedParams& p, const Misc* M, const Shape& sh,
                                              uint32_t tO, int c0, int used, int parity, bool whole, float* part,
                                              int d, bool store) {
    float o[K];
#pragma unroll
    for (int c = 0; c < K; ++c) o[c] = 0.f;
    for (int st = 0; st < used; ++st) {
        float x[K];
        const int unit = sh.wide ? 2 * st + (c0 >> 5) : st;
        tmem_ldn<K>(tO + sh.accum(st) + (uint32_t)c0, x);
#pragma unroll
        for (int c = 0; c < K; ++c) o[c] = fmaf(x[c], M->fac[unit][(c0 + c) & 31], o[c]);
    }
    if (!store) return;
#pragma unroll
    for (int c = 0; c < K; ++c) {
        const int64_t at = M->row_at[parity][c0 + c];
        if (at < 0) continue;
        if (whole)
            p.out[(size_t)at * HD + d] = __bfloat16_as_ushort(__float2bfloat16_rn(o[c]));
        else
            part[2 * kRowTile + (c0 + c) * HD + d] = o[c];
    }
}

// One segment's key tiles of unit u, COLS of its rows; then the streams'
// results are joined and written.  Every thread of all units walks the same
// barriers even after a wait ran out (the results are then not stored), so
// that no named barrier is left waiting.
template <int HD, bool F8, int COLS>
__device__ __forceinline__ void soft_segment(const PagedParams& p, const SegInfo& sg, Misc* M, uint8_t* smem,
                                             uint32_t tmem, int u, SoftState& st) {
    using C = Cfg<HD, F8>;
    volatile WaitState* ab = &M->wst;
    const Shape sh(sg.rows);
    const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int tr = wq * 32 + lane;                            // key of the tile; head_dim index of O^T
    const int bar = 1 + u, parity = st.seg & 1;
    const int stream = sh.stream_of(u), coff = sh.wide ? (u & 1) * kUnitRows : 0;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lanes + sh.scores<F8>(stream) + (uint32_t)coff;
    const uint32_t tO = tmem + lanes + C::kColO;
    uint8_t* P = smem + C::kOffP + u * C::kPBytes;
    const PlanInput& pl = p.plan;

    // this unit's rows
    const int qb = st.seg % C::kQ;
    if (F8) mbar_wait(&M->q_full[qb], (st.seg / C::kQ) & 1u, ab);
    if (tr < COLS) {
        const int64_t rho = (int64_t)sg.j * kRowTile + coff + tr;
        M->lim[u][tr] = coff + tr < sg.rows ? plan_seen(pl, sg.q, rho) : 0;
        M->nref[u][tr] = -kFloorRef;
        if (F8) M->qm[u][tr] = M->q_scale[qb][coff + tr];
    }
    if (u == 0 && tr < kRowTile) {
        const int64_t rho = (int64_t)sg.j * kRowTile + tr;
        const int i = (int)(rho / pl.group), g = (int)(rho - (int64_t)i * pl.group);
        M->row_at[parity][tr] = tr < sg.rows ? (int64_t)(sg.q.a + i) * p.heads + (int64_t)sg.h * pl.group + g : -1;
    }
    named_sync(bar, 128);
    if (F8 && lane == 0) mbar_arrive(&M->q_empty[qb]);        // the row scales are copied

    uint64_t l2[COLS / 2];
#pragma unroll
    for (int c = 0; c < COLS / 2; ++c) l2[c] = 0;
    const int lim0 = plan_seen(pl, sg.q, (int64_t)sg.j * kRowTile);   // the first row sees the fewest keys
    const int n = sg.n, t0 = sg.t0;

    for (int i = stream; i < n; i += sh.streams) {
        const int key = (t0 + i) * kKeyTile + tr;
        const bool edge = (t0 + i + 1) * kKeyTile > lim0;  // some row does not see the whole tile
        float mul = p.scale2, vs = 1.f;
        if (F8) {
            const uint32_t at = st.line + (uint32_t)i;
            const int s = (int)(at % C::kScMod);
            mbar_wait(&M->c_full[s], (at / C::kScMod) & 1u, ab);
            const int bp = min(1 << p.page_log2, kKeyTile), pitch = max(bp * 4, 128);
            const uint8_t* sc = smem + C::kOffSc + s * C::kScBytes + (tr / bp) * pitch + (tr % bp) * 4;
            mul *= *reinterpret_cast<const float*>(sc);
            vs = *reinterpret_cast<const float*>(sc + C::kScBytes / 2);
            __syncwarp();
            // a wide tile's scales are read by two units
            if (lane == 0) mbar_arrive(&M->c_empty[s]);
            if (!sh.wide && lane == 0) mbar_arrive(&M->c_empty[s]);
        }
        mbar_wait(&M->s_full[u], st.tiles & 1u, ab);
        tc_fence_after();

        // base-2 scores, minus the rows' references if `rel`
        float t[COLS];
        const uint64_t mul2 = pack2(mul, mul);
        auto load_scores = [&](auto rel) {
            tmem_ldn<COLS>(tS, t);
            auto minus_ref = [&](int c) {
                if constexpr (!decltype(rel)::value) return uint64_t(0);
                const float2 r = *reinterpret_cast<const float2*>(&M->nref[u][c]);
                return pack2(r.x, r.y);
            };
            if constexpr (F8) {
                const uint64_t k16 = pack2(0.0625f, 0.0625f);
#pragma unroll
                for (int h = 0; h < COLS; h += 16) {
                    float lo[16];
                    tmem_ldn<16>(tS + (uint32_t)(sh.cols + h), lo);
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        const uint64_t s = mul2x(fma2(pack2(lo[c], lo[c + 1]), k16, pack2(t[h + c], t[h + c + 1])), mul2);
                        const float2 qm = *reinterpret_cast<const float2*>(&M->qm[u][h + c]);
                        unpack2(fma2(s, pack2(qm.x, qm.y), minus_ref(h + c)), t[h + c], t[h + c + 1]);
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < COLS; c += 2)
                    unpack2(fma2(pack2(t[c], t[c + 1]), mul2, minus_ref(c)), t[c], t[c + 1]);
            }
            if (edge) {
#pragma unroll
                for (int c = 0; c < COLS; ++c)
                    if (key >= M->lim[u][c]) t[c] = -INFINITY;
            }
        };
        for (bool raised = false;; raised = true) {
            load_scores(std::true_type{});
            if (raised) break;
            float top = t[0];
#pragma unroll
            for (int c = 1; c < COLS; ++c) top = fmaxf(top, t[c]);
            if (!named_any(bar, 128, top > kLazy)) break;
            // raise the references to the largest scores so far, which happens
            // once (scores of 2^28 and more round by more than the threshold)
            load_scores(std::false_type{});
            float mine = 0.f;
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                const float mx = redux_max(t[c]);
                if (lane == c) mine = mx;
            }
            if (lane < COLS) M->red[u][wq][lane] = mine;
            named_sync(bar, 128);
            if (tr < COLS) {
                const float old = -M->nref[u][tr];
                const float ref = fmaxf(fmaxf(fmaxf(M->red[u][0][tr], M->red[u][1][tr]),
                                              fmaxf(M->red[u][2][tr], M->red[u][3][tr])), old);
                M->nref[u][tr] = -ref;
                M->fac[u][tr] = ex2_approx(old - ref);
            }
            named_sync(bar, 128);
#pragma unroll
            for (int c = 0; c < COLS; c += 2) {
                const float2 f = *reinterpret_cast<const float2*>(&M->fac[u][c]);
                l2[c / 2] = mul2x(l2[c / 2], pack2(f.x, f.y));
            }
            if (i >= sh.streams) {                            // the accumulator holds earlier tiles
                mbar_wait(&M->pv_done[u], (st.tiles - 1u) & 1u, ab);
                tc_fence_after();
                const uint32_t at = tO + sh.accum(stream) + (uint32_t)coff;
#pragma unroll
                for (int ch = 0; ch < COLS / 16; ++ch) {
                    float o[16];
                    tmem_ldn<16>(at + ch * 16, o);
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] *= M->fac[u][ch * 16 + c];
                    tmem_st16(at + ch * 16, o);
                }
                tmem_st_wait();
            }
        }
        // the P buffer is free once this unit's previous product is done
        if (st.tiles > 0) mbar_wait(&M->pv_done[u], (st.tiles - 1u) & 1u, ab);
        ++st.tiles;
        const uint64_t vs2 = pack2(vs, vs);
#pragma unroll
        for (int c8 = 0; c8 < COLS / 8; ++c8) {
            uint32_t pk[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int k = c8 * 8 + 2 * c;
                float a = ex2_approx(t[k]), b = ex2_approx(t[k + 1]);
                uint64_t w = pack2(a, b);
                l2[k / 2] = add2(l2[k / 2], w);
                if (F8) {
                    unpack2(mul2x(w, vs2), a, b);
                    if (edge) {
                        // a hidden key's weight stays 0 whatever its place holds as a scale
                        if (t[k] == -INFINITY) a = 0.f;
                        if (t[k + 1] == -INFINITY) b = 0.f;
                    }
                }
                // weights become bf16 for the product with V (half a step: 2^-9 of
                // each weight's binade); the sums keep them in float32
                const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                pk[c] = reinterpret_cast<const uint32_t&>(h);
            }
            *reinterpret_cast<uint4*>(P + c8 * (kKeyTile * 16) + tr * 16) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        if constexpr (F8) {
            // Widen V's e4m3 codes, 16 at a time; two units share a wide tile.
            // (The widened tile two before this one has been multiplied, and so
            // has whatever the loaded tile's place held before.)
            const uint32_t at = st.line + (uint32_t)i;
            const int d = (int)(at % C::kWMod), s = (int)(at % C::kV);
            mbar_wait(&M->w_empty[d], ((at / C::kWMod) & 1u) ^ 1u, ab);
            mbar_wait(&M->v_full[s], (at / C::kV) & 1u, ab);
            const uint8_t* src = smem + C::kOffV + (size_t)s * C::kLoadBytes;
            uint8_t* dst = smem + C::kOffW + (size_t)d * C::kTileBytes;
            constexpr int kPieces = kKeyTile * HD / 16, kPer = HD / 16;
            const int step = sh.wide ? 256 : 128;
#pragma unroll 2
            for (int x = coff * 4 + tr; x < kPieces; x += step) {
                const uint4 v = *reinterpret_cast<const uint4*>(src + x * 16);
                const uint2 a = e4m3x4_to_bf16x4(v.x), b = e4m3x4_to_bf16x4(v.y);
                const uint2 c = e4m3x4_to_bf16x4(v.z), e = e4m3x4_to_bf16x4(v.w);
                const int row = x / kPer, c0 = (x % kPer) * 2;
                uint8_t* rowp = dst + (c0 / 8) * C::kHalfBytes + row * 128;
                const int c8 = c0 & 7, sw = row & 7;
                // lanes of the second half write their pieces in the other order: no bank conflicts
                const bool flip = c0 >= 8;
                const uint4 lo = make_uint4(a.x, a.y, b.x, b.y), hi = make_uint4(c.x, c.y, e.x, e.y);
                *reinterpret_cast<uint4*>(rowp + ((c8 + (flip ? 1 : 0)) ^ sw) * 16) = flip ? hi : lo;
                *reinterpret_cast<uint4*>(rowp + ((c8 + (flip ? 0 : 1)) ^ sw) * 16) = flip ? lo : hi;
            }
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M->p_full[u]);
    }
    st.line += (uint32_t)n;
    ++st.seg;

    // the units' sums, then one factor per row and stream
    {
        float x[COLS];
#pragma unroll
        for (int c = 0; c < COLS; c += 2) unpack2(l2[c / 2], x[c], x[c + 1]);
        const float sum = lane_sums<COLS>(x);
        if (lane < COLS) M->red[u][wq][lane] = sum;
    }
    if (st.tiles > 0) mbar_wait(&M->pv_done[u], (st.tiles - 1u) & 1u, ab);
    tc_fence_after();
    named_sync(5, kUnits * 128);
    const bool whole = n == sg.tiles;
    float* part = p.part + (size_t)(blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * piece_floats(HD);
    const bool store = !ab->abort;
    const int used = min(n, sh.streams);                      // streams with an accumulator
    if (u == 0 && tr < sh.cols) {
        const int c = tr & 31;
        auto unit = [&](int s) { return sh.wide ? 2 * s + (tr >> 5) : s; };
        float m = kFloorRef;
        for (int s = 0; s < used; ++s) m = fmaxf(m, -M->nref[unit(s)][c]);
        float sum = 0.f;
        for (int s = 0; s < used; ++s) {
            const float* r = &M->red[unit(s)][0][c];
            const float l = r[0] + r[kUnitRows] + r[2 * kUnitRows] + r[3 * kUnitRows];
            const float f = ex2_approx(-M->nref[unit(s)][c] - m);
            sum = fmaf(l, f, sum);
            M->fac[unit(s)][c] = f;
        }
        const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
        for (int s = 0; s < used; ++s) M->fac[unit(s)][c] *= inv;
        const int64_t at = M->row_at[parity][tr];
        if (store && whole && p.lse && at >= 0) p.lse[at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
        if (store && !whole) {
            part[tr] = m;
            part[kRowTile + tr] = sum;
        }
    }
    if (u == 0 && tr == 0 && t0 == 0 && !whole) {             // the last segment of the span
        const int spans = plan_spans(M->total, (int)gridDim.x);
        const int64_t last_tile = plan_cut(M->total, (int)blockIdx.x + 1, spans) - n + sg.tiles - 1;
        p.desc[blockIdx.x] = JoinDesc{sg.r, sg.j, sg.h, plan_owner(M->total, last_tile, spans)};
    }
    named_sync(5, kUnits * 128);
    const bool mine = store && tr < HD;
    if (COLS == 32 && sh.wide)
        store_columns<HD, 16>(p, M, sh, tO, u * 16, used, parity, whole, part, tr, mine);
    else
        store_columns<HD, COLS / 4>(p, M, sh, tO, u * (COLS / 4), used, parity, whole, part, tr, mine);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&M->o_free);
}

template <int HD, bool F8>
__global__ void __launch_bounds__(kThreads, 1)
    attn_paged_kernel(const __grid_constant__ Maps maps, const PagedParams p) {
    using C = Cfg<HD, F8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc* M = reinterpret_cast<Misc*>(smem + C::kOffMisc);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PlanInput& pl = p.plan;
    const int cta = (int)blockIdx.x;
    pdl_launch_dependents();

    // ---------------- this CTA's span
    if (cta == 0) check_requests(pl.q_off, pl.kv_len, pl.R, pl.T, pl.most, p.ws);
    const int per = (pl.R + kThreads - 1) / kThreads;
    const int r0 = min((int)threadIdx.x * per, pl.R), r1 = min(r0 + per, pl.R);
    int64_t sum = 0;
    for (int r = r0; r < r1; ++r) sum += plan_request_tiles(pl, r);
    int64_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) M->scan[warp] = upto;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kK; ++i) {
            mbar_init(&M->k_full[i], 1);
            mbar_init(&M->k_empty[i], 1);
        }
        for (int i = 0; i < C::kV; ++i) {
            mbar_init(&M->v_full[i], 1);
            mbar_init(&M->v_empty[i], 1);
        }
        for (int i = 0; i < C::kW; ++i) mbar_init(&M->w_empty[i], 1);
        for (int i = 0; i < C::kSc; ++i) {
            mbar_init(&M->c_full[i], 1);
            mbar_init(&M->c_empty[i], 8);
        }
        for (int i = 0; i < C::kQ; ++i) {
            mbar_init(&M->q_full[i], 32);
            mbar_init(&M->q_empty[i], F8 ? 1 + 4 * kUnits : 1);
        }
        for (int i = 0; i < kUnits; ++i) {
            mbar_init(&M->s_full[i], 1);
            mbar_init(&M->p_full[i], 4);
            mbar_init(&M->pv_done[i], 1);
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(&M->seg_full[i], 1);
            mbar_init(&M->seg_empty[i], kReaders);
        }
        mbar_init(&M->o_free, 4 * kUnits);
        mbar_init(&M->done, 1);
        M->wst.abort = 0;
        M->wst.limit = ws_wait_limit(p.ws);
        fence_mbar_init();
        p.desc[cta] = JoinDesc{-1, 0, 0, 0};
    }
    __syncthreads();
    int64_t base = upto - sum, total = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) base += M->scan[i];
        total += M->scan[i];
    }
    const int spans = plan_spans(total, (int)gridDim.x);
    if (cta >= spans) return;                                 // the same for every thread of the CTA
    const int64_t begin = plan_cut(total, cta, spans), end = plan_cut(total, cta + 1, spans);
    if (base <= begin && begin < base + sum) {
        int64_t at = base;
        int r = r0;
        for (;; ++r) {
            const int64_t t = plan_request_tiles(pl, r);
            if (begin < at + t) break;
            at += t;
        }
        M->start_r = r;
        M->start_skip = begin - at;
    }
    if (threadIdx.x == 0) M->total = total;
    if (warp == 1) tmem_alloc(&M->tmem, C::kTmem);
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
        if (!__all_sync(0xffffffffu, mbar_wait(&M->seg_full[at], (nseg / kSegs) & 1u, ab))) return false;
        sg = M->seg[at];
        return sg.rows > 0;
    };
    auto done_segment = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&M->seg_empty[nseg % kSegs]);
        ++nseg;
    };

    const int bp = min(1 << p.page_log2, kKeyTile);           // tokens of a page inside one tile
    const int ppt = kKeyTile / bp;                            // pages of a tile

    if (warp == 0) {
        // ---------------- producer
        const uint64_t once = policy_evict_first(), again = policy_evict_normal();
        uint32_t nk = 0, nv = 0;
        const int pg = lane & 7, sub = lane >> 3;
        bool ok = true;
        for (; ok && next_segment(); done_segment()) {
            // more than one row tile of a request reads its keys again
            const uint64_t pol = (int64_t)sg.q.q_len * pl.group > kRowTile ? again : once;
            const int32_t* table = p.page_table + (size_t)sg.r * p.max_pages;
            const int n = sg.n, ahead = min(Shape(sg.rows).streams, n);
            // the page of this lane's part of key tile i (-1: past the keys)
            auto page_of = [&](int i) {
                const int64_t tok = (int64_t)(sg.t0 + i) * kKeyTile + pg * bp;
                if (i >= n || pg >= ppt || tok >= sg.keys) return -1;
                int id = __ldg(table + (tok >> p.page_log2));
                if (id < 0 || id >= p.n_pages) {
                    raise_status(p.ws, kStatBadPage);
                    id = p.n_pages;                           // past the tensor: zeros
                }
                return id;
            };
            auto issue = [&](bool is_v, int i, int id) {
                const uint32_t g = is_v ? nv++ : nk++;
                const int ring = is_v ? C::kV : C::kK, s = (int)(g % ring);
                uint64_t *full = is_v ? M->v_full : M->k_full, *empty = is_v ? M->v_empty : M->k_empty;
                ok = ok && __all_sync(0xffffffffu, mbar_wait(&empty[s], ((g / ring) & 1u) ^ 1u, ab));
                const int c = (int)(g % C::kScMod);
                if (F8 && !is_v)
                    ok = ok && __all_sync(0xffffffffu, mbar_wait(&M->c_empty[c], ((g / C::kScMod) & 1u) ^ 1u, ab));
                if (!ok) {
                    (is_v ? nv : nk) -= 1;
                    return;
                }
                const int pages = __popc(__ballot_sync(0xffffffffu, id >= 0 && lane < 8));
                const int tok0 = ((sg.t0 + i) * kKeyTile) & ((1 << p.page_log2) - 1);   // place inside a 256-token page
                const int x = (sg.h << p.page_log2) + (ppt == 1 ? tok0 : 0);
                if (lane == 0) {
                    mbar_expect_tx(&full[s], (uint32_t)(pages * bp * (F8 ? HD : HD * 2)));
                    if (F8 && !is_v) mbar_expect_tx(&M->c_full[c], (uint32_t)(pages * bp * 8));
                }
                __syncwarp();
                if (id < 0) return;
                if (sub < (F8 ? 1 : C::kHalves))
                    tma_load_3d(smem + (is_v ? C::kOffV : 0) + (size_t)s * C::kLoadBytes + (F8 ? 0 : sub * C::kHalfBytes) +
                                    pg * bp * (F8 ? HD : 128),
                                is_v ? &maps.v : &maps.k, &full[s], sub * 64, x, id, pol);
                else if (F8 && !is_v && sub < 3)
                    tma_load_2d(smem + C::kOffSc + c * C::kScBytes + (sub - 1) * (C::kScBytes / 2) + pg * max(bp * 4, 128),
                                sub == 1 ? &maps.ks : &maps.vs, &M->c_full[c], x, id, pol);
            };
            // K runs `ahead` tiles before V; ids[k] is the page of tile i + k
            int ids[6];
#pragma unroll
            for (int k = 0; k < 5; ++k) ids[k] = page_of(k);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < ahead) issue(false, k, ids[k]);
            for (int i = 0; ok && i < n; ++i) {
                ids[5] = page_of(i + 5);
                if (i + ahead < n)
                    issue(false, i + ahead, ahead == 4 ? ids[4] : (ahead == 3 ? ids[3] : (ahead == 2 ? ids[2] : ids[1])));
                issue(true, i, ids[0]);
#pragma unroll
                for (int k = 0; k < 5; ++k) ids[k] = ids[k + 1];
            }
        }
        // every copy that was issued lands before the CTA may leave
        __syncwarp();
        if (ab->abort && lane == 0) {
            for (uint32_t k = nk > C::kK ? nk - C::kK : 0; k < nk; ++k)
                mbar_wait_for(&M->k_full[k % C::kK], (k / C::kK) & 1u, ab->limit);
            for (uint32_t k = nv > C::kV ? nv - C::kV : 0; k < nv; ++k)
                mbar_wait_for(&M->v_full[k % C::kV], (k / C::kV) & 1u, ab->limit);
            if (F8)
                for (uint32_t k = nk > (uint32_t)C::kSc ? nk - C::kSc : 0; k < nk; ++k)
                    mbar_wait_for(&M->c_full[k % C::kScMod], (k / C::kScMod) & 1u, ab->limit);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer
        constexpr uint32_t a_lbo = HD == 128 ? C::kHalfBytes : 0;   // head_dim 64: rows 64..127 repeat 0..63
        uint32_t nk = 0, nv = 0, np = 0;                      // np: parity of each unit's next p_full, by bit
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t par) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, par, ab));
            tc_fence_after();
            return ok;
        };
        for (; ok && next_segment(); done_segment()) {
            const int n = sg.n;
            const Shape sh(sg.rows);
            const uint32_t id_qk = F8 ? idesc_e4m3_f32(128, 2 * sh.cols) : idesc_bf16_f32(128, sh.cols, false, false);
            const uint32_t id_pv = idesc_bf16_f32(128, sh.cols, true, true);
            const int qb = nseg % C::kQ;
            const uint8_t* qt = smem + C::kOffQ + qb * C::kQBytes;
            auto scores = [&](int i) {
                const int s = (int)(nk % C::kK), st = i % sh.streams;
                if (!wait(&M->k_full[s], (nk / C::kK) & 1u)) return;
                if (lane == 0) {
                    const uint8_t* kt = smem + (size_t)s * C::kLoadBytes;
                    const uint32_t d = tmem + sh.scores<F8>(st);
                    if (F8) {
#pragma unroll
                        for (int kk = 0; kk < HD / 32; ++kk)
                            umma_f8(d, desc_f8<HD>(kt + kk * 32), desc_f8<HD>(qt + kk * 32), id_qk, kk ? 1u : 0u);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk)
                            umma_bf16(d, smem_desc_sw128(kt + (kk / 4) * C::kHalfBytes + (kk % 4) * 32, 16, 1024),
                                      smem_desc_sw128(qt + (kk / 4) * (kRowTile * 128) + (kk % 4) * 32, 16, 1024), id_qk,
                                      kk ? 1u : 0u);
                    }
                    umma_commit(&M->k_empty[s]);
                    umma_commit(&M->s_full[sh.wide ? 2 * st : st]);
                    if (sh.wide) umma_commit(&M->s_full[2 * st + 1]);
                    if (i == n - 1) umma_commit(&M->q_empty[qb]);
                }
                __syncwarp();
                ++nk;
            };
            if (!wait(&M->q_full[qb], (nseg / C::kQ) & 1u)) break;
            for (int i = 0; ok && i < n && i < sh.streams; ++i) scores(i);
            for (int i = 0; ok && i < n; ++i) {
                const int st = i % sh.streams, u0 = sh.wide ? 2 * st : st;
                if (!wait(&M->p_full[u0], (np >> u0) & 1u)) break;
                if (sh.wide && !wait(&M->p_full[u0 + 1], (np >> (u0 + 1)) & 1u)) break;
                np ^= (sh.wide ? 3u : 1u) << u0;
                if (i + sh.streams < n) scores(i + sh.streams);
                if (i == 0 && nseg > 0) wait(&M->o_free, (nseg - 1u) & 1u);
                // bf16: the V tile as it was loaded; e4m3: the widened one, which
                // p_full covers, as it does the end of the reads of the loaded one
                const int s = (int)(nv % C::kV), d = (int)(nv % C::kWMod);
                if (!F8) wait(&M->v_full[s], (nv / C::kV) & 1u);
                if (!ok) break;
                uint8_t* vt = smem + (F8 ? C::kOffW + (size_t)d * C::kTileBytes : C::kOffV + (size_t)s * C::kTileBytes);
                const int valid = sg.keys - (sg.t0 + i) * kKeyTile;
                if (!F8 && valid < kKeyTile) {
                    // rows past the last key hold whatever the pages or this buffer held
                    for (int x = max(valid, 0) * 8 + lane; x < kKeyTile * 8; x += 32)
#pragma unroll
                        for (int hf = 0; hf < C::kHalves; ++hf)
                            *reinterpret_cast<uint4*>(vt + hf * C::kHalfBytes + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async();
                    __syncwarp();
                }
                if (lane == 0) {
                    const uint8_t* pt = smem + C::kOffP + u0 * C::kPBytes;
#pragma unroll
                    for (int kk = 0; kk < kKeyTile / 16; ++kk)
                        umma_bf16(tmem + C::kColO + sh.accum(st), smem_desc_sw128(vt + kk * 2048, a_lbo, 1024),
                                  smem_desc_plain(pt + kk * 256, 128, kKeyTile * 16), id_pv,
                                  (i >= sh.streams || kk) ? 1u : 0u);
                    if (F8) mbar_arrive(&M->v_empty[s]);
                    umma_commit(F8 ? &M->w_empty[d] : &M->v_empty[s]);
                    umma_commit(&M->pv_done[u0]);
                    if (sh.wide) umma_commit(&M->pv_done[u0 + 1]);
                }
                __syncwarp();
                ++nv;
            }
        }
        // the tensor core is idle before its memory is given back
        if (lane == 0) {
            umma_commit(&M->done);
            mbar_wait_for(&M->done, 0, ab->limit);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---------------- Q rows
        const uint64_t pol = policy_evict_normal();
        constexpr int kLanes = HD / 8;                        // 8 values per lane
        for (; next_segment(); done_segment()) {
            const int qb = nseg % C::kQ;
            if (!__all_sync(0xffffffffu, mbar_wait(&M->q_empty[qb], ((nseg / C::kQ) & 1u) ^ 1u, ab))) break;
            const int cols = Shape(sg.rows).cols;
            uint8_t* qt = smem + C::kOffQ + qb * C::kQBytes;
            for (int x = lane; x < cols * kLanes; x += 32) {
                const int row = x / kLanes, c = x % kLanes;
                const int64_t rho = (int64_t)sg.j * kRowTile + row;
                const int i = (int)(rho / pl.group), gq = (int)(rho - (int64_t)i * pl.group);
                const bool in = row < sg.rows;
                const uint16_t* src = in ? p.q + (int64_t)(sg.q.a + i) * p.q_stride +
                                               ((int64_t)sg.h * pl.group + gq) * HD + c * 8
                                         : p.q;
                if (!F8) {
                    cp_async16_zf(qt + (c / 8) * (kRowTile * 128) + row * 128 + ((c ^ row) & 7) * 16, src, in ? 16u : 0u,
                                  pol);
                    continue;
                }
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (in) v = __ldg(reinterpret_cast<const uint4*>(src));
                uint2 hi, lo;
                const float s = split_e4m3<kLanes>(v, hi, lo);
                const int at = swz_f8<HD>(row, c / 2) + (c & 1) * 8, at_lo = swz_f8<HD>(cols + row, c / 2) + (c & 1) * 8;
                *reinterpret_cast<uint2*>(qt + at) = hi;
                *reinterpret_cast<uint2*>(qt + at_lo) = lo;
                if (c == 0) M->q_scale[qb][row] = s;
            }
            if (!F8) cp_async_wait_all();
            fence_proxy_async();
            mbar_arrive(&M->q_full[qb]);
        }
    } else if (warp == 3) {
        // ---------------- segments
        if (lane == 0) {
            Cursor cur;
            cur.start(pl, M->start_r, M->start_skip, end - begin);
            Segment s;
            for (uint32_t k = 0;; ++k) {
                const int at = k % kSegs;
                const bool more = cur.next(pl, s);
                if (!mbar_wait(&M->seg_empty[at], ((k / kSegs) & 1u) ^ 1u, ab)) break;
                SegInfo& o = M->seg[at];
                o.rows = more ? s.rows : 0;
                if (more) {
                    o.r = s.r;
                    o.j = s.j;
                    o.h = s.h;
                    o.t0 = s.t0;
                    o.n = s.t1 - s.t0;
                    o.tiles = s.tiles;
                    o.keys = s.keys;
                    o.q = s.q;
                }
                mbar_arrive(&M->seg_full[at]);
                if (!more) break;
            }
        }
    } else {
        // ---------------- softmax
        const int u = (warp - 4) >> 2;
        SoftState st = {0, 0, 0};
        for (;; ++nseg) {
            const int at = nseg % kSegs;
            const bool got = mbar_wait(&M->seg_full[at], (nseg / kSegs) & 1u, ab);
            // all units agree on whether there is a segment; what the one
            // before left in shared memory is no longer read
            if (named_any(5, kUnits * 128, !got)) break;
            const SegInfo& s = M->seg[at];
            if (s.rows == 0) break;
            if (s.rows <= 16)
                soft_segment<HD, F8, 16>(p, s, M, smem, tmem, u, st);
            else
                soft_segment<HD, F8, 32>(p, s, M, smem, tmem, u, st);
            __syncwarp();
            if (lane == 0) mbar_arrive(&M->seg_empty[at]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && M->wst.abort) raise_status(p.ws, kStatTimeout);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmem);
    }
}

// ------------------------------------------------------------------ join
// Block (c, y) joins 8 rows of the item that starts in CTA c's span and ends
// in a later one: a warp per row, pieces in the order of the keys.
template <int HD>
__global__ void __launch_bounds__(256) attn_paged_join(const PagedParams p, int grid) {
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

template <int HD, bool F8>
cudaError_t launch(const Maps& maps, const PagedParams& p, int grid, cudaStream_t s) {
    const size_t smem = smem_bytes<HD, F8>();
    cudaError_t e = cudaFuncSetAttribute(attn_paged_kernel<HD, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    prof_begin(kPAttnPaged, s);
    e = launch_kernel(attn_paged_kernel<HD, F8>, dim3(grid), dim3(kThreads), smem, s, false, maps, p);
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
    p.q = static_cast<const uint16_t*>(q);
    p.q_stride = q_stride;
    p.plan = PlanInput{b.q_off, b.kv_len, b.R, b.T, n_heads / c.n_kv_heads, c.n_kv_heads, (int64_t)b.max_pages * c.page};
    p.page_table = b.page_table;
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
    const bool f8 = c.dtype == DSPARK_E4M3;
    const cuuint64_t hd = (cuuint64_t)c.head_dim, rows = (cuuint64_t)c.n_kv_heads * c.page, pages = (cuuint64_t)c.n_pages;
    const cuuint32_t bp = (cuuint32_t)(c.page < kKeyTile ? c.page : kKeyTile);
    const cuuint64_t es = f8 ? 1 : 2;
    const cuuint64_t dims[3] = {hd, rows, pages}, str[2] = {hd * es, rows * hd * es};
    const cuuint32_t box[3] = {f8 ? (cuuint32_t)hd : 64u, bp, 1};
    const CUtensorMapDataType dt = f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    // e4m3: K feeds the tensor core in rows of head_dim bytes, V the widening
    const CUtensorMapSwizzle swz_k = f8 && hd == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    const CUtensorMapSwizzle swz_v = f8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
    bool ok = make_tensor_map(&maps.k, dt, 3, c.k, dims, str, box, swz_k) &&
              make_tensor_map(&maps.v, dt, 3, c.v, dims, str, box, swz_v);
    if (f8) {
        const cuuint64_t sd[2] = {rows, pages}, ss[1] = {rows * 4};
        const cuuint32_t sb[2] = {bp, 1};
        ok = ok && make_tensor_map(&maps.ks, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, c.k_scale, sd, ss, sb, CU_TENSOR_MAP_SWIZZLE_NONE) &&
             make_tensor_map(&maps.vs, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, c.v_scale, sd, ss, sb, CU_TENSOR_MAP_SWIZZLE_NONE);
    } else {
        maps.ks = maps.k;
        maps.vs = maps.v;
    }
    if (!ok) return cudaErrorInvalidValue;
    if (c.head_dim == 64) return f8 ? launch<64, true>(maps, p, grid, s) : launch<64, false>(maps, p, grid, s);
    return f8 ? launch<128, true>(maps, p, grid, s) : launch<128, false>(maps, p, grid, s);
}

}  // namespace dspark
