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
//   warp 2      Q rows of the next item, by cp.async
//   warps 4-11  two softmax warpgroups; warpgroup w takes every second key
//               tile with its own reference, sum and accumulator, so that one
//               exponentiates while the other's products run.  Thread = key,
//               registers = rows.  The reference of a row is raised only when
//               a score exceeds it by more than 2^8 (a vote per tile; p <= 2^8
//               is far inside bf16 and float32), so a tile costs no maximum
//               over its keys.
//   warps 12-19 (e4m3 caches) widen the raw tiles to bf16 exactly
//
// Keys a row must not see get weight 0 by selection, not by multiplication;
// V rows past the item's last key are zeroed in shared memory, since 0 times
// a stale NaN would be NaN.
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

template <int HD, bool F8>
struct Cfg {
    static constexpr int kTileBytes = kKeyTile * HD * 2;                   // a K or V tile as bf16
    static constexpr int kHalves = HD / 64;                                // 128-byte swizzle atoms of a row
    static constexpr int kHalfBytes = kKeyTile * 128;
    static constexpr int kTiles = F8 ? (HD == 128 ? 3 : 5) : (HD == 128 ? 5 : 10);   // ring of bf16 tiles
    static constexpr int kRaw = F8 ? (HD == 128 ? 4 : 8) : 0;              // ring of e4m3 tiles
    static constexpr int kRawBytes = kKeyTile * HD;
    static constexpr int kSc = F8 ? 4 : 0;                                 // ring of scale tiles (K, V)
    static constexpr int kScBytes = 2048;                                  // 2 x 128 scales, 16-token pages at 128-byte pitch
    static constexpr int kRawMod = kRaw ? kRaw : 1, kScMod = kSc ? kSc : 1;   // divisors (unused without e4m3)
    static constexpr int kPBytes = kKeyTile * kRowTile * 2;
    static constexpr int kQBytes = kRowTile * HD * 2;
    static constexpr int kCvtWarps = F8 ? 8 : 0;
    static constexpr int kThreads = 32 * (12 + kCvtWarps);
    static constexpr int kBars = 2 * kTiles + 2 * kRaw + 2 * kSc + 2 + 6 + 1 + 1;
    static constexpr int kOffRaw = kTiles * kTileBytes;
    static constexpr int kOffP = kOffRaw + kRaw * kRawBytes;
    static constexpr int kOffQ = kOffP + 2 * kPBytes;
    static constexpr int kOffSc = kOffQ + kQBytes;
    static constexpr int kOffMisc = kOffSc + kSc * kScBytes;
};

struct Misc {
    int64_t row_at[2][kRowTile];       // element offset of a row in out (-1: no row), per warpgroup
    int lim[2][kRowTile];              // keys a row sees
    float ref[2][kRowTile];            // reference m
    float fac[2][kRowTile];            // factor of a raised reference, then of the join
    float red[2][4][kRowTile];         // per-warp maxima, then sums
    float tot_m[kRowTile], tot_l[kRowTile];
    int64_t scan[32];
    int64_t total;
    int64_t start_skip;
    int start_r;
    uint32_t tmem;
    WaitState wst;
};

template <int HD, bool F8>
constexpr size_t smem_bytes() {
    return 1024 + Cfg<HD, F8>::kOffMisc + sizeof(Misc) + 8 * Cfg<HD, F8>::kBars + 64;
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

// Sums over the 32 lanes of N = 16, 32 or 64 values per lane; lane i gets the
// sums of values i (N = 32), i and i + 32 (N = 64), i % 16 (N = 16).
template <int N>
__device__ __forceinline__ void lane_sums(float (&v)[N]) {
    const int lane = threadIdx.x & 31;
    if constexpr (N == 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
    }
    constexpr int kBlocks = N == 64 ? 2 : 1;
    constexpr int kTop = N == 16 ? 8 : 16;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        float* x = v + 32 * b;
#pragma unroll
        for (int o = kTop; o > 0; o >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < o; ++i) {
                const float keep = up ? x[i + o] : x[i], give = up ? x[i] : x[i + o];
                x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        }
    }
}

// ------------------------------------------------------------------ softmax
struct SoftState {
    uint32_t s_seen, pv_seen;          // completed waits on s_full and pv_done of this warpgroup
};

struct Bars {
    uint64_t *t_full, *t_empty, *r_full, *r_empty, *c_full, *c_empty, *q_full, *q_empty, *s_full, *p_full, *pv_done,
        *o_free, *done;
};

template <int HD, bool F8>
__device__ __forceinline__ Bars carve_bars(uint8_t* at) {
    using C = Cfg<HD, F8>;
    Bars b;
    b.t_full = reinterpret_cast<uint64_t*>(at);
    b.t_empty = b.t_full + C::kTiles;
    b.r_full = b.t_empty + C::kTiles;
    b.r_empty = b.r_full + C::kRaw;
    b.c_full = b.r_empty + C::kRaw;
    b.c_empty = b.c_full + C::kSc;
    b.q_full = b.c_empty + C::kSc;
    b.q_empty = b.q_full + 1;
    b.s_full = b.q_empty + 1;
    b.p_full = b.s_full + 2;
    b.pv_done = b.p_full + 2;
    b.o_free = b.pv_done + 2;
    b.done = b.o_free + 1;
    return b;
}

// One segment's key tiles of warpgroup w, for up to 16 NCH rows; then the
// warpgroups' results are joined and written.  Every thread of both
// warpgroups walks the same barriers even after a wait ran out (the results
// are then not stored), so that no named barrier is left waiting.
template <int HD, bool F8, int NCH>
__device__ __forceinline__ void soft_segment(const PagedParams& p, const Segment& sg, const Bars& B, Misc* M,
                                             uint8_t* smem, uint32_t tmem, int w, uint32_t& sc_at, SoftState& st,
                                             int piece, int64_t span_end, int spans) {
    using C = Cfg<HD, F8>;
    constexpr int N = 16 * NCH;
    volatile WaitState* ab = &M->wst;
    const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int tr = wq * 32 + lane;                            // key of the tile; head_dim index of O^T
    const int bar = 1 + w;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lanes + (uint32_t)(w * kRowTile);
    const uint32_t tO = tmem + lanes + 2 * kRowTile;
    uint8_t* P = smem + C::kOffP + w * C::kPBytes;
    const PlanInput& pl = p.plan;

    named_sync(bar, 128);                                     // the previous segment's rows are no longer read
    if (tr < N) {
        const int64_t rho = (int64_t)sg.j * kRowTile + tr;
        const bool in = tr < sg.rows;
        const int i = (int)(rho / pl.group), g = (int)(rho - (int64_t)i * pl.group);
        M->lim[w][tr] = in ? plan_seen(pl, sg.q, rho) : 0;
        M->row_at[w][tr] = in ? ((int64_t)(sg.q.a + i) * p.heads + (int64_t)sg.h * pl.group + g) : -1;
        M->ref[w][tr] = kFloorRef;
    }
    named_sync(bar, 128);

    float l[N];
#pragma unroll
    for (int c = 0; c < N; ++c) l[c] = 0.f;
    const int lim0 = plan_seen(pl, sg.q, (int64_t)sg.j * kRowTile);   // the first row sees the fewest keys
    const int n = sg.t1 - sg.t0;

    for (int i = w; i < n; i += 2) {
        const int key = (sg.t0 + i) * kKeyTile + tr;
        const bool edge = (sg.t0 + i + 1) * kKeyTile > lim0;  // some row does not see the whole tile
        float mul = p.scale2, vs = 1.f;
        if (F8) {
            const uint32_t at = sc_at + (uint32_t)i;
            const int s = (int)(at % C::kScMod);
            mbar_wait(&B.c_full[s], (at / C::kScMod) & 1u, ab);
            const int bp = p.page_log2 >= 7 ? kKeyTile : (1 << p.page_log2), pitch = max(bp * 4, 128);
            const uint8_t* sc = smem + C::kOffSc + s * C::kScBytes + (tr / bp) * pitch + (tr % bp) * 4;
            mul *= *reinterpret_cast<const float*>(sc);
            vs = *reinterpret_cast<const float*>(sc + C::kScBytes / 2);
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.c_empty[s]);
        }
        mbar_wait(&B.s_full[w], st.s_seen & 1u, ab);
        ++st.s_seen;
        tc_fence_after();

        auto load_scores = [&](int ch, float (&s)[16]) {
            tmem_ld16(tS + ch * 16, s);
#pragma unroll
            for (int c = 0; c < 16; ++c) s[c] *= mul;
            if (edge) {
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    if (key >= M->lim[w][ch * 16 + c]) s[c] = -INFINITY;
            }
        };
        // does any score exceed its row's reference by more than kLazy bits?
        bool over = false;
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
            float s[16];
            load_scores(ch, s);
#pragma unroll
            for (int c = 0; c < 16; ++c) over |= s[c] > M->ref[w][ch * 16 + c] + kLazy;
        }
        if (named_any(bar, 128, over)) {
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch) {
                float s[16];
                load_scores(ch, s);
                float mine = 0.f;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const float mx = redux_max(s[c]);
                    if (lane == c) mine = mx;
                }
                if (lane < 16) M->red[w][wq][ch * 16 + lane] = mine;
            }
            named_sync(bar, 128);
            if (tr < N) {
                const float old = M->ref[w][tr];
                const float mx = fmaxf(fmaxf(fmaxf(M->red[w][0][tr], M->red[w][1][tr]),
                                             fmaxf(M->red[w][2][tr], M->red[w][3][tr])), old);
                M->fac[w][tr] = ex2_approx(old - mx);
                M->ref[w][tr] = mx;
            }
            named_sync(bar, 128);
#pragma unroll
            for (int c = 0; c < N; ++c) l[c] *= M->fac[w][c];
            if (i >= 2) {                                     // the accumulator holds earlier tiles
                mbar_wait(&B.pv_done[w], (st.pv_seen - 1u) & 1u, ab);
                tc_fence_after();
#pragma unroll
                for (int ch = 0; ch < NCH; ++ch) {
                    float o[16];
                    tmem_ld16(tO + (uint32_t)(w * kRowTile + ch * 16), o);
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] *= M->fac[w][ch * 16 + c];
                    tmem_st16(tO + (uint32_t)(w * kRowTile + ch * 16), o);
                }
                tmem_st_wait();
            }
        }
        // the P buffer is free once this warpgroup's previous product is done
        if (st.pv_seen > 0) mbar_wait(&B.pv_done[w], (st.pv_seen - 1u) & 1u, ab);
        ++st.pv_seen;
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
            float s[16];
            load_scores(ch, s);
            uint32_t pk[8];
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
                float a = ex2_approx(s[c] - M->ref[w][ch * 16 + c]);
                float b = ex2_approx(s[c + 1] - M->ref[w][ch * 16 + c + 1]);
                l[ch * 16 + c] += a;
                l[ch * 16 + c + 1] += b;
                if (F8) {
                    // a weight of 0 stays 0 whatever a place without a key holds as its scale
                    a = edge && a == 0.f ? 0.f : a * vs;
                    b = edge && b == 0.f ? 0.f : b * vs;
                }
                // weights become bf16 for the product with V (half a step: 2^-9 of
                // each weight's binade); the sum l keeps them in float32
                const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                pk[c / 2] = reinterpret_cast<const uint32_t&>(h);
            }
            uint8_t* dst = P + (2 * ch) * (kKeyTile * 16) + tr * 16;
            *reinterpret_cast<uint4*>(dst) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            *reinterpret_cast<uint4*>(dst + kKeyTile * 16) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.p_full[w]);
    }
    sc_at += (uint32_t)n;

    // the warpgroups' sums, then one factor per row and warpgroup
    lane_sums<N>(l);
    if (N == 64) {
        M->red[w][wq][lane] = l[0];
        M->red[w][wq][lane + 32] = l[32 % N];
    } else if (lane < N) {
        M->red[w][wq][lane] = l[0];
    }
    if (st.pv_seen > 0) mbar_wait(&B.pv_done[w], (st.pv_seen - 1u) & 1u, ab);
    tc_fence_after();
    named_sync(3, 256);
    const bool whole = sg.t0 == 0 && sg.t1 == sg.tiles;
    float* part = p.part + (size_t)piece * piece_floats(HD);
    const bool store = !ab->abort;
    if (w == 0 && tr < N) {
        const float m0 = M->ref[0][tr], m1 = M->ref[1][tr], m = fmaxf(m0, m1);
        const float l0 = M->red[0][0][tr] + M->red[0][1][tr] + M->red[0][2][tr] + M->red[0][3][tr];
        const float l1 = M->red[1][0][tr] + M->red[1][1][tr] + M->red[1][2][tr] + M->red[1][3][tr];
        const float f0 = ex2_approx(m0 - m), f1 = ex2_approx(m1 - m);
        const float sum = l0 * f0 + l1 * f1;
        const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
        M->tot_m[tr] = f0 * inv;
        M->tot_l[tr] = f1 * inv;
        if (store && whole && p.lse && M->row_at[0][tr] >= 0)
            p.lse[M->row_at[0][tr]] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
        if (store && !whole) {
            part[tr] = m;
            part[kRowTile + tr] = sum;
        }
    }
    if (w == 0 && tr == 0 && sg.t0 == 0 && !whole) {
        const int64_t last_tile = span_end - (sg.t1 - sg.t0) + sg.tiles - 1;
        p.desc[blockIdx.x] = JoinDesc{sg.r, sg.j, sg.h, plan_owner(M->total, last_tile, spans)};
    }
    named_sync(3, 256);
    const bool two = n > 1;                                   // warpgroup 1 has an accumulator
#pragma unroll
    for (int ch = 0; ch < NCH; ++ch) {
        if ((NCH == 1 ? 0 : (ch & 1)) != w) continue;
        float o[16];
        tmem_ld16(tO + ch * 16, o);
#pragma unroll
        for (int c = 0; c < 16; ++c) o[c] *= M->tot_m[ch * 16 + c];
        if (two) {
            float o1[16];
            tmem_ld16(tO + kRowTile + ch * 16, o1);
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] = fmaf(o1[c], M->tot_l[ch * 16 + c], o[c]);
        }
        if (tr < HD && store) {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const int64_t at = M->row_at[w][ch * 16 + c];
                if (at < 0) continue;
                if (whole)
                    p.out[(size_t)at * HD + tr] = __bfloat16_as_ushort(__float2bfloat16_rn(o[c]));
                else
                    part[2 * kRowTile + (ch * 16 + c) * HD + tr] = o[c];
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(B.o_free);
}

template <int HD, bool F8>
__global__ void __launch_bounds__(Cfg<HD, F8>::kThreads, 1)
    attn_paged_kernel(const __grid_constant__ Maps maps, const PagedParams p) {
    using C = Cfg<HD, F8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc* M = reinterpret_cast<Misc*>(smem + C::kOffMisc);
    const Bars B = carve_bars<HD, F8>(smem + C::kOffMisc + ((sizeof(Misc) + 15) & ~size_t(15)));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PlanInput& pl = p.plan;
    const int cta = (int)blockIdx.x;
    pdl_launch_dependents();

    // ---------------- this CTA's span
    if (cta == 0) check_requests(pl.q_off, pl.kv_len, pl.R, pl.T, pl.most, p.ws);
    const int per = (pl.R + C::kThreads - 1) / C::kThreads;
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
        for (int i = 0; i < C::kTiles; ++i) {
            mbar_init(&B.t_full[i], F8 ? C::kCvtWarps : 1);
            mbar_init(&B.t_empty[i], 1);
        }
        for (int i = 0; i < C::kRaw; ++i) {
            mbar_init(&B.r_full[i], 1);
            mbar_init(&B.r_empty[i], C::kCvtWarps);
        }
        for (int i = 0; i < C::kSc; ++i) {
            mbar_init(&B.c_full[i], 1);
            mbar_init(&B.c_empty[i], 4);
        }
        mbar_init(B.q_full, 32);
        mbar_init(B.q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B.s_full[i], 1);
            mbar_init(&B.p_full[i], 4);
            mbar_init(&B.pv_done[i], 1);
        }
        mbar_init(B.o_free, 8);
        mbar_init(B.done, 1);
        M->wst.abort = 0;
        M->wst.limit = ws_wait_limit(p.ws);
        fence_mbar_init();
        p.desc[cta] = JoinDesc{-1, 0, 0, 0};
    }
    __syncthreads();
    int64_t base = upto - sum, total = 0;
    for (int i = 0; i < C::kThreads / 32; ++i) {
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
    if (warp == 1) tmem_alloc(&M->tmem, 256);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = M->tmem;
    volatile WaitState* ab = &M->wst;
    Cursor cur;
    cur.start(pl, M->start_r, M->start_skip, end - begin);
    Segment sg;

    const int bp = min(1 << p.page_log2, kKeyTile);           // tokens of a page inside one tile
    const int ppt = kKeyTile / bp;                            // pages of a tile

    if (warp == 0) {
        // ---------------- producer
        const uint64_t once = policy_evict_first(), again = policy_evict_normal();
        constexpr int kRing = F8 ? C::kRaw : C::kTiles;
        uint64_t* full = F8 ? B.r_full : B.t_full;
        uint64_t* empty = F8 ? B.r_empty : B.t_empty;
        constexpr int kStage = F8 ? C::kRawBytes : C::kTileBytes;
        uint8_t* ring = smem + (F8 ? C::kOffRaw : 0);
        uint32_t g = 0, sc = 0;
        const int pg = lane & 7, sub = lane >> 3;
        bool ok = true;
        while (ok && cur.next(pl, sg)) {
            // more than one row tile of a request reads its keys again
            const uint64_t pol = (int64_t)sg.q.q_len * pl.group > kRowTile ? again : once;
            const int32_t* table = p.page_table + (size_t)sg.r * p.max_pages;
            // the page of this lane's part of key tile i (-1: past the keys)
            auto page_of = [&](int i) {
                const int64_t tok = (int64_t)(sg.t0 + i) * kKeyTile + pg * bp;
                if (i >= sg.t1 - sg.t0 || pg >= ppt || tok >= sg.keys) return -1;
                int id = __ldg(table + (tok >> p.page_log2));
                if (id < 0 || id >= p.n_pages) {
                    raise_status(p.ws, kStatBadPage);
                    id = p.n_pages;                           // past the tensor: zeros
                }
                return id;
            };
            auto issue = [&](bool is_v, int i, int id) {
                const int s = (int)(g % kRing);
                ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], ((g / kRing) & 1u) ^ 1u, ab));
                if (!ok) return;
                const int n = __popc(__ballot_sync(0xffffffffu, id >= 0 && lane < 8));
                const int tok0 = (sg.t0 + i) * kKeyTile & ((1 << p.page_log2) - 1);   // place inside a 256-token page
                const int x = (sg.h << p.page_log2) + (ppt == 1 ? tok0 : 0);
                uint8_t* dst = ring + (size_t)s * kStage + pg * (F8 ? bp * HD : bp * 128);
                if (F8 && !is_v) {
                    const int c = (int)(sc % C::kScMod);
                    ok = __all_sync(0xffffffffu, mbar_wait(&B.c_empty[c], ((sc / C::kScMod) & 1u) ^ 1u, ab));
                    if (!ok) return;
                    if (lane == 0) mbar_expect_tx(&B.c_full[c], (uint32_t)(n * bp * 8));
                    __syncwarp();
                    if ((sub == 1 || sub == 2) && id >= 0)
                        tma_load_2d(smem + C::kOffSc + c * C::kScBytes + (sub - 1) * (C::kScBytes / 2) + pg * max(bp * 4, 128),
                                    sub == 1 ? &maps.ks : &maps.vs, &B.c_full[c], x, id, pol);
                    ++sc;
                }
                if (lane == 0) mbar_expect_tx(&full[s], (uint32_t)(n * bp * (F8 ? HD : HD * 2)));
                __syncwarp();
                if (id >= 0 && sub < (F8 ? 1 : C::kHalves))
                    tma_load_3d(dst + (F8 ? 0 : sub * C::kHalfBytes), is_v ? &maps.v : &maps.k, &full[s], sub * 64, x, id,
                                pol);
                ++g;
            };
            const int n = sg.t1 - sg.t0;
            int id0 = page_of(0), id1 = page_of(1), id2 = page_of(2);
            issue(false, 0, id0);
            if (ok && n > 1) issue(false, 1, id1);
            for (int i = 0; ok && i < n; ++i) {
                const int id3 = page_of(i + 3);
                if (i + 2 < n) issue(false, i + 2, id2);
                if (ok) issue(true, i, id0);
                id0 = id1;
                id1 = id2;
                id2 = id3;
            }
        }
        // every copy that was issued lands before the CTA may leave
        __syncwarp();
        if (ab->abort && lane == 0) {
            for (uint32_t k = g > kRing ? g - kRing : 0; k < g; ++k)
                mbar_wait_for(&full[k % kRing], (k / kRing) & 1u, ab->limit);
            if (F8)
                for (uint32_t k = sc > (uint32_t)C::kSc ? sc - C::kSc : 0; k < sc; ++k)
                    mbar_wait_for(&B.c_full[k % C::kScMod], (k / C::kScMod) & 1u, ab->limit);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer
        constexpr uint32_t a_lbo = HD == 128 ? C::kHalfBytes : 0;   // head_dim 64: rows 64..127 repeat 0..63
        uint32_t g = 0, np[2] = {0, 0}, nseg = 0;
        bool ok = true;
        while (ok && cur.next(pl, sg)) {
            const int n = sg.t1 - sg.t0;
            const int cols = sg.rows <= 16 ? 16 : (sg.rows <= 32 ? 32 : 64);
            const uint32_t id_qk = idesc_bf16_f32(128, cols, false, false);
            const uint32_t id_pv = idesc_bf16_f32(128, cols, true, true);
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                const bool k = __all_sync(0xffffffffu, mbar_wait(bar, parity, ab));
                tc_fence_after();
                return k;
            };
            auto scores = [&](int i) {
                const int s = (int)(g % C::kTiles);
                if (!wait(&B.t_full[s], (g / C::kTiles) & 1u)) return false;
                if (lane == 0) {
                    const uint8_t* kt = smem + (size_t)s * C::kTileBytes;
                    const uint8_t* qt = smem + C::kOffQ;
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk)
                        umma_bf16(tmem + (uint32_t)((i & 1) * kRowTile),
                                  smem_desc_sw128(kt + (kk / 4) * C::kHalfBytes + (kk % 4) * 32, 16, 1024),
                                  smem_desc_sw128(qt + (kk / 4) * (kRowTile * 128) + (kk % 4) * 32, 16, 1024), id_qk,
                                  kk ? 1u : 0u);
                    umma_commit(&B.t_empty[s]);
                    umma_commit(&B.s_full[i & 1]);
                    if (i == n - 1) umma_commit(B.q_empty);
                }
                __syncwarp();
                ++g;
                return true;
            };
            ok = wait(B.q_full, nseg & 1u) && scores(0) && (n == 1 || scores(1));
            for (int i = 0; ok && i < n; ++i) {
                const int w = i & 1;
                ok = wait(&B.p_full[w], np[w]++ & 1u);
                if (ok && i + 2 < n) ok = scores(i + 2);
                const int s = (int)(g % C::kTiles);
                ok = ok && wait(&B.t_full[s], (g / C::kTiles) & 1u);
                if (ok && i == 0 && nseg > 0) ok = wait(B.o_free, (nseg - 1u) & 1u);
                if (!ok) break;
                uint8_t* vt = smem + (size_t)s * C::kTileBytes;
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
                    const uint8_t* pt = smem + C::kOffP + w * C::kPBytes;
#pragma unroll
                    for (int kk = 0; kk < kKeyTile / 16; ++kk)
                        umma_bf16(tmem + (uint32_t)(2 * kRowTile + w * kRowTile),
                                  smem_desc_sw128(vt + kk * 2048, a_lbo, 1024),
                                  smem_desc_plain(pt + kk * 256, 128, kKeyTile * 16), id_pv, (i >= 2 || kk) ? 1u : 0u);
                    umma_commit(&B.t_empty[s]);
                    umma_commit(&B.pv_done[w]);
                }
                __syncwarp();
                ++g;
            }
            ++nseg;
        }
        // the tensor core is idle before its memory is given back
        if (lane == 0) {
            umma_commit(B.done);
            mbar_wait_for(B.done, 0, ab->limit);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---------------- Q rows
        uint32_t nseg = 0;
        const uint64_t pol = policy_evict_normal();
        while (cur.next(pl, sg)) {
            if (!__all_sync(0xffffffffu, mbar_wait(B.q_empty, (nseg & 1u) ^ 1u, ab))) break;
            const int cols = sg.rows <= 16 ? 16 : (sg.rows <= 32 ? 32 : 64);
            constexpr int kChunks = HD / 8;                   // 16-byte pieces of a row
            for (int x = lane; x < cols * kChunks; x += 32) {
                const int row = x / kChunks, c = x % kChunks;
                const int64_t rho = (int64_t)sg.j * kRowTile + row;
                const int i = (int)(rho / pl.group), gq = (int)(rho - (int64_t)i * pl.group);
                const bool in = row < sg.rows;
                const uint16_t* src = in ? p.q + (int64_t)(sg.q.a + i) * p.q_stride +
                                               ((int64_t)sg.h * pl.group + gq) * HD + c * 8
                                         : p.q;
                cp_async16_zf(smem + C::kOffQ + (c / 8) * (kRowTile * 128) + row * 128 + ((c ^ row) & 7) * 16, src,
                              in ? 16u : 0u, pol);
            }
            cp_async_wait_all();
            fence_proxy_async();
            mbar_arrive(B.q_full);
            ++nseg;
        }
    } else if (warp >= 4 && warp < 12) {
        // ---------------- softmax
        const int w = (warp - 4) >> 2;
        uint32_t sc_at = 0;
        SoftState st = {0, 0};
        while (cur.next(pl, sg)) {
            const int piece = cta * 2 + (sg.t0 == 0 ? 1 : 0);
            if (sg.rows <= 16)
                soft_segment<HD, F8, 1>(p, sg, B, M, smem, tmem, w, sc_at, st, piece, end, spans);
            else if (sg.rows <= 32)
                soft_segment<HD, F8, 2>(p, sg, B, M, smem, tmem, w, sc_at, st, piece, end, spans);
            else
                soft_segment<HD, F8, 4>(p, sg, B, M, smem, tmem, w, sc_at, st, piece, end, spans);
        }
    } else if (F8 && warp >= 12) {
        // ---------------- e4m3 -> bf16, one 16-byte piece (16 values) at a time
        const int ct = threadIdx.x - 12 * 32;
        constexpr int kPieces = kKeyTile * HD / 16, kPer = HD / 16;
        uint32_t g = 0;
        bool ok = true;
        while (ok && cur.next(pl, sg)) {
            for (int i = 0; ok && i < 2 * (sg.t1 - sg.t0); ++i, ++g) {
                const int s = (int)(g % C::kRawMod), d = (int)(g % C::kTiles);
                ok = mbar_wait(&B.r_full[s], (g / C::kRawMod) & 1u, ab) &&
                     mbar_wait(&B.t_empty[d], ((g / C::kTiles) & 1u) ^ 1u, ab);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint8_t* src = smem + C::kOffRaw + (size_t)s * C::kRawBytes;
                uint8_t* dst = smem + (size_t)d * C::kTileBytes;
#pragma unroll
                for (int x = ct; x < kPieces; x += C::kCvtWarps * 32) {
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
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&B.r_empty[s]);
                    mbar_arrive(&B.t_full[d]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && M->wst.abort) raise_status(p.ws, kStatTimeout);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
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
    e = launch_kernel(attn_paged_kernel<HD, F8>, dim3(grid), dim3(Cfg<HD, F8>::kThreads), smem, s, false, maps, p);
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
    const CUtensorMapSwizzle swz = f8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
    bool ok = make_tensor_map(&maps.k, dt, 3, c.k, dims, str, box, swz) &&
              make_tensor_map(&maps.v, dt, 3, c.v, dims, str, box, swz);
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
