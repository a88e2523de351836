// attn_prompt.cu -- causal attention over whole prompts, packed one after
// another (sm_103a: TMA, tcgen05, TMEM).
//
// A row is one token of one query head; a row tile is 128 rows: the whole
// group of query heads that share a key-value head, for 128 / group tokens
// (groups that do not divide 128 leave a few rows unused).  So a tile of keys
// is loaded once for the group, short sequences fill the tensor core's rows
// with heads, and causality wastes less than a tile of 128 tokens would.
//
//   S = Q K^T [128 rows x 128 keys]   P = 2^(S c - m)   O += P V
//
// One persistent CTA per SM works on two row tiles at a time, so that one
// tile's softmax runs beside the other's products:
//   warp 0      TMA producer: the two Q tiles, then K and V tiles into a ring
//   warps 1, 2  MMA issuers, one per row tile s: S_s and O_s in TMEM, P_s over
//               S_s's columns (bf16).  (One warp for both left the tensor core
//               idle for a third of the time, between its waits.)
//   warp 3      zeroes the rows of the last V tile that no row of the item may
//               see (0 times another sequence's NaN would be NaN)
//   warps 4-11  softmax, one warpgroup per row tile, one row per thread: no
//               exchange between threads; the reference m is raised only when
//               a score exceeds it by more than 2^8, so the accumulator is
//               rescaled once or twice per item rather than at every tile
// Items (a pair of row tiles and a key-value head) are handed out from the
// longest to the shortest, forwards and backwards over the CTAs in turn.
//
// 0 times a NaN or an infinity is NaN, so such a value in V would reach the rows
// before its token too.  A CTA that has stored a row that is not finite goes over
// its items once more: warp 3 then takes what is not finite out of the V tiles
// that some row of the item does not see the whole of, and adds it to the rows
// that do see it when they are stored.  (Looking through those tiles in the
// first place made 12001 tokens 12 % and packed prompts 20 % slower: warp 3's
// loads wait behind the tensor core's reads of shared memory.)
//
// Bound by the tensor core and the softmax beside it: the two products of a
// tile of 128 x 128 scores take it about 1024 cycles at head_dim 128.
// Measured (GB300): one sequence of 12001 tokens, 32 heads over 8 of 128: 789
// to 847 us, 1.39 to 1.50 PFLOP/s of the causal half (a plain bf16 product of
// 8192^3 runs at 1.90 in a burst and 1.73 under the power cap), of 64: 676 us; 16
// sequences of 100 to 4000 tokens: 590 to 612 us, 1.11 to 1.15 PFLOP/s.  (Taking
// a quarter of the exponentials from the XU pipe to a polynomial on the FMA pipe
// cost 18 %: its instructions cost more than the pipe it relieves.)
#include <cfloat>

#include <cuda.h>

#include "kernels.h"
#include "kv.cuh"
#include "profile.h"
#include "sm100.cuh"

namespace dspark {

namespace {

constexpr int kRows = 128;              // rows of a row tile
constexpr int kKeys = 128;              // keys of a key tile
constexpr int kThreads = 384;
constexpr int kPlanThreads = 1024;
constexpr float kFloorRef = -1e30f;
constexpr float kLazy = 8.f;

template <int HD>
struct Cfg {
    static constexpr int kHalves = HD / 64;
    static constexpr int kHalfBytes = 128 * 128;             // 128 rows of one 128-byte swizzle atom
    static constexpr int kTileBytes = kHalves * kHalfBytes;
    static constexpr int kStages = HD == 128 ? 5 : 8;        // ring of K and V tiles
    static constexpr int kOffQ = kStages * kTileBytes;
    static constexpr int kOffMisc = kOffQ + 2 * kTileBytes;
};

struct Bars {
    uint64_t full[8], empty[8];
    uint64_t q_full[2], q_empty[2], s_full[2], s_read[2], p_full[2][2], pv_done[2], o_free[2];
    // A V tile for warp 3 to clear, asked for by the issuers of the row tiles s
    // that use it, and, by ring place, cleared.  (One barrier for both issuers'
    // requests took the request of an item that one of them had reached for the
    // item before it; one per issuer for the answers could be two phases ahead
    // of its reader.  Either ended in a wait that ran out, with many sequences of
    // a few tiles.)
    uint64_t asked[2], fixed[8];
    uint64_t done;
};

struct Misc {
    Bars b[2];                          // the first and the second time over the items
    WaitState wst;
    uint32_t tmem;
    uint32_t again;                     // a stored row was not finite
    // warp 3's own: first token (from the item's first) whose V holds a
    // +infinity, a -infinity (a NaN counts as both) in each of the head's values
    uint16_t since[2][128];
    // this CTA's entry and the number of entries, where there is no list (a
    // CTA past the last entry has none, and the workspace no room for one)
    int2 own;
    int entries;
};

template <int HD>
constexpr size_t smem_bytes() {
    constexpr size_t bytes = 1024 + Cfg<HD>::kOffMisc + sizeof(Misc);
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    return bytes;
}

struct Params {
    const int32_t* seq_off;
    const int2* list;                   // (sequence, pair of row tiles), longest first
    const int* count;                   // entries of the list
    int most;                           // entries that the workspace holds
    int single;                         // no CTA gets a second item: each finds its own entry
    uint16_t* out;
    float* lse;
    void* ws;
    int B, T, heads, kv_heads, group, toks;   // toks: tokens of a row tile
    float scale2;                       // scale log2(e)
};

// Pairs of row tiles of a sequence.
__device__ __forceinline__ int pairs_of(const Params& p, int b) {
    const RowRange r = row_range(p.seq_off, b, p.T);
    return (r.b - r.a + 2 * p.toks - 1) / (2 * p.toks);
}

// The list of (sequence, pair of row tiles) entries in descending order of
// their length (the tile's place in its sequence), by a counting sort over
// 1024 classes of places.  Entries of a class stand in any order: each item's
// result depends on the item alone.
__global__ void __launch_bounds__(kPlanThreads) attn_prompt_plan(Params p, int2* list, int* count) {
    pdl_launch_dependents();
    using u64 = unsigned long long;                          // overlapping sequences (bad offsets) can sum to anything
    __shared__ u64 at[kPlanThreads];
    __shared__ u64 warp_sum_sh[32];
    __shared__ int most;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) most = 1;
    at[tid] = 0;
    __syncthreads();
    check_requests(p.seq_off, nullptr, p.B, p.T, 0, p.ws);
    const int pair = 2 * p.toks;
    int mine = 1;
    for (int b = tid; b < p.B; b += kPlanThreads) {
        const RowRange r = row_range(p.seq_off, b, p.T);
        mine = max(mine, (r.b - r.a + pair - 1) / pair);
    }
    if (mine > 1) atomicMax(&most, mine);
    __syncthreads();
    const int64_t n_class = most;
    auto each = [&](auto f) {
        for (int b = warp; b < p.B; b += kPlanThreads / 32) {
            const RowRange r = row_range(p.seq_off, b, p.T);
            const int n = (r.b - r.a + pair - 1) / pair;
            for (int t = lane; t < n; t += 32) f(b, t, kPlanThreads - 1 - (int)((int64_t)t * kPlanThreads / n_class));
        }
    };
    each([&](int, int, int c) { atomicAdd(&at[c], u64(1)); });
    __syncthreads();
    // exclusive sums over the classes
    const u64 v = at[tid];
    u64 upto = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) warp_sum_sh[warp] = upto;
    __syncthreads();
    u64 base = 0;
    for (int i = 0; i < warp; ++i) base += warp_sum_sh[i];
    at[tid] = base + upto - v;
    if (tid == kPlanThreads - 1) *count = (int)min(base + upto, (u64)p.most);
    __syncthreads();
    // only offsets that decrease can give more entries than the workspace has
    // room for (sequences that overlap); what does not fit is left out
    each([&](int b, int t, int c) {
        const u64 k = atomicAdd(&at[c], u64(1));
        if (k < (u64)p.most) list[k] = make_int2(b, t);
    });
}

struct Item {
    int a, len;                         // the sequence's first row and its tokens
    int tok0;                           // first token of row tile 0
    int h;                              // key-value head
    int n0, n1;                         // key tiles of each row tile (0: no rows)
    int keys;                           // keys that the item's last token sees
    // first V tile to clear: with rows past the item's keys (none: tiles()), or,
    // the second time, with a key that some row of the item does not see
    __device__ __forceinline__ int edge(bool second) const {
        return second ? min((tok0 + 1) / kKeys, tiles() - 1) : keys / kKeys;
    }
    __device__ __forceinline__ int n(int s) const { return s ? n1 : n0; }
    __device__ __forceinline__ int tiles() const { return max(n0, n1); }
};

// Entry k of the list in the order of the sequences, and how many there are,
// by one warp.
__device__ __forceinline__ int2 entry_of(const Params& p, int64_t k, int64_t& count) {
    const int lane = threadIdx.x & 31;
    int2 e = make_int2(0, 0);
    count = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        const int n = b < p.B ? pairs_of(p, b) : 0;
        int64_t upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        const int64_t first = count + upto - n;
        const uint32_t m = __ballot_sync(0xffffffffu, first <= k && k < first + n);
        if (m) {
            e.x = b0 + __ffs(m) - 1;
            e.y = (int)(k - __shfl_sync(0xffffffffu, first, __ffs(m) - 1));
        }
        count += __shfl_sync(0xffffffffu, upto, 31);
    }
    return e;
}

__device__ __forceinline__ bool get_item(const Params& p, const Misc* M, int64_t total, int round, Item& it) {
    const int64_t n = gridDim.x, c = blockIdx.x;
    const int64_t k = (int64_t)round * n + ((round & 1) ? n - 1 - c : c);
    if (k >= total) return false;
    // the list was written by the kernel before this one
    const int2 e = p.single ? M->own : __ldcg(p.list + k / p.kv_heads);
    it.h = (int)(k % p.kv_heads);
    const RowRange r = row_range(p.seq_off, e.x, p.T);
    it.a = __shfl_sync(0xffffffffu, r.a, 0);                  // the same in every lane, as the compiler now knows
    it.len = __shfl_sync(0xffffffffu, r.b, 0) - it.a;
    it.tok0 = __shfl_sync(0xffffffffu, e.y, 0) * 2 * p.toks;
    auto tiles = [&](int first) {
        return first < it.len ? (min(it.len, first + p.toks) + kKeys - 1) / kKeys : 0;
    };
    it.n0 = tiles(it.tok0);
    it.n1 = tiles(it.tok0 + p.toks);
    it.keys = min(it.len, it.tok0 + 2 * p.toks);
    return true;
}

// 32 columns of this thread's lane, without waiting; tmem_ready() on the same
// registers makes them usable.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
#define DSPARK_PIN32(v)                                                                                              \
    "+f"((v)[0]), "+f"((v)[1]), "+f"((v)[2]), "+f"((v)[3]), "+f"((v)[4]), "+f"((v)[5]), "+f"((v)[6]), "+f"((v)[7]), \
        "+f"((v)[8]), "+f"((v)[9]), "+f"((v)[10]), "+f"((v)[11]), "+f"((v)[12]), "+f"((v)[13]), "+f"((v)[14]),      \
        "+f"((v)[15]), "+f"((v)[16]), "+f"((v)[17]), "+f"((v)[18]), "+f"((v)[19]), "+f"((v)[20]), "+f"((v)[21]),    \
        "+f"((v)[22]), "+f"((v)[23]), "+f"((v)[24]), "+f"((v)[25]), "+f"((v)[26]), "+f"((v)[27]), "+f"((v)[28]),    \
        "+f"((v)[29]), "+f"((v)[30]), "+f"((v)[31])
// Waits for this thread's tensor-memory loads; v is usable afterwards (the
// registers are operands, so no use of them can be scheduled before it).
__device__ __forceinline__ void tmem_ready(float* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : DSPARK_PIN32(v)::"memory");
}
__device__ __forceinline__ void tmem_pin(float* v) { asm volatile("" : DSPARK_PIN32(v)); }

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

struct Maps {
    CUtensorMap q, k, v;
};

template <int HD>
__device__ __forceinline__ void init_bars(Bars* B) {
    using C = Cfg<HD>;
    for (int i = 0; i < C::kStages; ++i) {
        mbar_init(&B->full[i], 1);
        mbar_init(&B->empty[i], 2);
        mbar_init(&B->fixed[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
        mbar_init(&B->q_full[s], 1);
        mbar_init(&B->q_empty[s], 1);
        mbar_init(&B->s_full[s], 1);
        mbar_init(&B->s_read[s], 4);
        mbar_init(&B->p_full[s][0], 4);
        mbar_init(&B->p_full[s][1], 4);
        mbar_init(&B->asked[s], 1);
        mbar_init(&B->pv_done[s], 1);
        mbar_init(&B->o_free[s], 4);
    }
    mbar_init(&B->done, 2);
    fence_mbar_init();
}

// One time over the CTA's items: warps 0 to 3.
template <int HD, bool kSecond>
__device__ __forceinline__ void few_roles(const Maps& maps, const Params& p, Misc* M, uint8_t* smem, uint32_t tmem,
                                          int64_t total, int warp, int lane) {
    using C = Cfg<HD>;
    Bars* B = &M->b[kSecond];
    volatile WaitState* ab = &M->wst;
    Item it;

    if (warp == 0) {
        // ---------------- producer
        const uint64_t pol_q = policy_evict_first(), pol_kv = policy_evict_last();
        uint32_t g = 0, st = 0, ph = 0, nq = 0, used = 0;     // tiles issued; the next ring place and its phase; Q's
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, wait_bar_here(bar, parity, ab)); };
        auto tile = [&](const CUtensorMap* m, int j) {
            wait(&B->empty[st], ph ^ 1u);
            if (!ok) return;
            if (elect_one()) {
                mbar_expect_tx(&B->full[st], (uint32_t)C::kTileBytes);
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf)
                    tma_load_3d(smem + st * C::kTileBytes + hf * C::kHalfBytes, m, &B->full[st], hf * 64, it.h,
                                it.a + j * kKeys, pol_kv);
            }
            __syncwarp();
            ++g;
            if (++st == C::kStages) {
                st = 0;
                ph ^= 1u;
            }
        };
        auto query = [&](int s) {
            if (!it.n(s)) return;
            wait(&B->q_empty[s], ((nq >> s) & 1u) ^ 1u);
            if (!ok) return;
            nq ^= 1u << s;
            used |= 1u << s;
            if (elect_one()) {
                mbar_expect_tx(&B->q_full[s], (uint32_t)(p.toks * p.group * HD * 2));
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf)
                    tma_load_3d(smem + C::kOffQ + s * C::kTileBytes + hf * C::kHalfBytes, &maps.q, &B->q_full[s], hf * 64,
                                it.h * p.group, it.a + it.tok0 + s * p.toks, pol_q);
            }
            __syncwarp();
        };
#pragma unroll 1
        for (int round = 0; ok && get_item(p, M, total, round, it); ++round) {
            const int n = it.tiles();
            query(0);
            tile(&maps.k, 0);
            query(1);
#pragma unroll 1
            for (int j = 0; ok && j < n; ++j) {
                if (j) tile(&maps.k, j);
                tile(&maps.v, j);
            }
        }
        // copies in flight land before the CTA may leave
        if (ab->abort && lane == 0) {
            for (uint32_t k = g > C::kStages ? g - C::kStages : 0; k < g; ++k)
                mbar_wait_for(&B->full[k % C::kStages], (k / C::kStages) & 1u, ab->limit);
            for (int s = 0; s < 2; ++s)
                if (used >> s & 1u) mbar_wait_for(&B->q_full[s], ((nq >> s) & 1u) ^ 1u, ab->limit);
        }
        __syncwarp();
    } else if (warp < 3) {
        // ---------------- MMA issuer of row tile s
        const int s = warp - 1;
        constexpr uint32_t id_qk = idesc_bf16_f32(128, 64, false, false);
        constexpr uint32_t id_pv = idesc_bf16_f32(128, HD, false, true);
        // descriptors of Q and of the first ring tile; others lie a constant number
        // of 16-byte units on (addresses stay inside the 14-bit field)
        const uint64_t dq = smem_desc_sw128(smem + C::kOffQ + s * C::kTileBytes, 16, 1024);
        const uint64_t dk = smem_desc_sw128(smem, 16, 1024);
        const uint64_t dv = smem_desc_sw128(smem, C::kHalfBytes, 1024);
        const uint32_t tS = tmem + (uint32_t)(s * 128), tO = tmem + (uint32_t)(256 + s * HD);
        uint32_t nq = 0, nr = 0, np = 0, no = 0;              // parities of the next waits
        uint32_t nfix = 0;                                    // the same for each ring place's `fixed`, by bit
        uint32_t st = 0, ph = 0;                              // ring place of the next tile, and its phase
        bool ok = true, started = false;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, wait_bar_here(bar, parity, ab));
            return ok;
        };
        auto next = [&]() {
            if (++st == C::kStages) {
                st = 0;
                ph ^= 1u;
            }
        };
        // Scores of 64 keys of the ring tile at `at`: half 1 goes to columns 64 to
        // 127 and may start as soon as the scores there before have been read,
        // half 0 to columns 0 to 63, over P, once P has been multiplied (the
        // tensor core runs a thread's MMAs in order).
        auto scores = [&](uint32_t at, int half, int j) {
            tc_fence_after();
            if (elect_one()) {
                const uint64_t b = dk + at * (C::kTileBytes / 16) + half * 512;
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t off = (kk / 4) * (C::kHalfBytes / 16) + (kk % 4) * 2;
                    umma_bf16(tS + half * 64, dq + off, b + off, id_qk, kk ? 1u : 0u);
                }
                if (!half) {
                    umma_commit(&B->s_full[s]);
                    umma_commit(&B->empty[at]);
                    if (j + 1 == it.n(s)) umma_commit(&B->q_empty[s]);
                }
            }
            __syncwarp();
        };
#pragma unroll 1
        for (int round = 0; ok && get_item(p, M, total, round, it); ++round) {
            const int n = it.tiles();
            if (it.n(s)) {
                if (!wait(&B->q_full[s], nq & 1u)) break;
                nq ^= 1u;
                // a last row tile's rows of the next sequence
                const int first = it.tok0 + s * p.toks;
                if (it.len - first < p.toks) {
                    uint8_t* qt = smem + C::kOffQ + s * C::kTileBytes;
#pragma unroll 1
                    for (int x = (it.len - first) * p.group * 8 + lane; x < p.toks * p.group * 8; x += 32)
#pragma unroll
                        for (int hf = 0; hf < C::kHalves; ++hf)
                            *reinterpret_cast<uint4*>(qt + hf * C::kHalfBytes + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async();
                    __syncwarp();
                }
            }
            if (!wait(&B->full[st], ph)) break;
            if (it.n(s)) {
                // (the item before it has been read and multiplied)
                scores(st, 1, 0);
                scores(st, 0, 0);
            } else if (lane == 0) {
                mbar_arrive(&B->empty[st]);
            }
            next();
#pragma unroll 1
            for (int j = 0; ok && j < n; ++j) {
                // V_j at st, K_{j+1} at the place after it
                const uint32_t vat = st, vph = ph;
                next();
                const uint32_t kat = st, kph = ph;
                if (j + 1 < n) next();
                if (j < it.n(s)) {
                    if (!wait(&B->s_read[s], nr & 1u)) break;
                    nr ^= 1u;
                    if (j + 1 < it.n(s)) {
                        if (!wait(&B->full[kat], kph)) break;
                        scores(kat, 1, j + 1);
                    }
                }
                if (!wait(&B->full[vat], vph)) break;
                const bool fix = j >= it.edge(kSecond);
                if (j < it.n(s)) {
                    // warp 3 starts while P is still being made
                    if (fix && lane == 0) mbar_arrive(&B->asked[s]);
                    if (j == 0) {
                        if (started) {                        // the item before has been stored
                            if (!wait(&B->o_free[s], no & 1u)) break;
                            no ^= 1u;
                        }
                        started = true;
                    }
                    if (fix && !wait(&B->fixed[vat], (nfix >> vat) & 1u)) break;
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {    // 64 keys at a time
                        if (!wait(&B->p_full[s][half], np & 1u)) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t b = dv + vat * (C::kTileBytes / 16) + half * 512;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_bf16_ts(tO, tS + half * 32 + kk * 8, b + kk * 128, id_pv, (j | half | kk) ? 1u : 0u);
                            if (half) {
                                umma_commit(&B->pv_done[s]);
                                umma_commit(&B->empty[vat]);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    np ^= 1u;
                    if (j + 1 < it.n(s)) scores(kat, 0, j + 1);
                } else if (lane == 0) {
                    mbar_arrive(&B->empty[vat]);
                }
                if (fix) nfix ^= 1u << vat;
                if (j + 1 < n && j + 1 >= it.n(s)) {          // a tile only the other row tile sees
                    if (!wait(&B->full[kat], kph)) break;
                    if (lane == 0) mbar_arrive(&B->empty[kat]);
                }
            }
        }
        // the tensor core is idle before its memory is given back
        if (elect_one()) {
            umma_commit(&B->done);
            mbar_wait_for(&B->done, 0, ab->limit);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ---------------- clear the last V tiles
        uint32_t g = 0;                                       // ring tiles before this item
        uint32_t asked = 0, stored = 0;                       // parity of each row tile's next request and store, by bit
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, wait_bar_here(bar, parity, ab));
            return ok;
        };
        constexpr int kPer = HD / 8;                          // 16-byte pieces of a row
        constexpr int kStep = 32 / kPer;                      // rows of a step: a lane keeps to one piece
        const int piece = lane % kPer, sub = lane / kPer;
#pragma unroll 1
        for (int round = 0; ok && get_item(p, M, total, round, it); ++round) {
            const int n = it.tiles();
            uint32_t add = 0;                                 // row tiles that the table matters to, by bit
#pragma unroll 1
            for (int j = it.edge(kSecond); j < n; ++j) {
                // the issuers that use the tile have seen it arrive (its parity alone
                // could be an earlier tile's), and the rows of the items before are stored
                const uint32_t vi = g + 2 * j + 1, vat = vi % C::kStages;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (j >= it.n(s)) continue;
                    wait(&B->asked[s], (asked >> s) & 1u);
                    asked ^= 1u << s;
                }
                if (!wait(&B->full[vat], (vi / C::kStages) & 1u)) break;
                uint8_t* vt = smem + vat * C::kTileBytes + (piece / 8) * C::kHalfBytes;
                auto at = [&](int row) { return reinterpret_cast<uint4*>(vt + row * 128 + ((piece ^ row) & 7) * 16); };
                const int valid = min(it.keys - j * kKeys, kKeys);
                if (kSecond) {
                    if (!add) {
#pragma unroll 1
                        for (int x = lane; x < 256; x += 32) (&M->since[0][0])[x] = 0xFFFFu;
                    }
                    // the lanes of a piece in turn: the table is theirs together
                    bool found = false;
#pragma unroll 1
                    for (int turn = 0; turn < kStep; ++turn) {
                        __syncwarp();
                        if (sub != turn) continue;
                        // every row sees the keys up to the item's first token
#pragma unroll 1
                        for (int row = max(it.tok0 + 1 - j * kKeys, 0); row < valid; ++row) {
                            if (row % kStep != turn) continue;
                            const uint4 w = *at(row);
                            const uint32_t top =
                                __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
                            if (max(top & 0xFFFFu, top >> 16) < 0x7F80u) continue;
                            found = true;
                            uint16_t* x = reinterpret_cast<uint16_t*>(at(row));
                            const uint16_t tok = (uint16_t)(j * kKeys + row - it.tok0);
#pragma unroll 1
                            for (int e = 0; e < 8; ++e) {
                                const uint32_t v = x[e];
                                if ((v & 0x7F80u) != 0x7F80u) continue;
                                uint16_t* plus = &M->since[0][piece * 8 + e];
                                uint16_t* minus = &M->since[1][piece * 8 + e];
                                if ((v & 0x7Fu) || !(v & 0x8000u)) *plus = min(*plus, tok);
                                if ((v & 0x7Fu) || (v & 0x8000u)) *minus = min(*minus, tok);
                                x[e] = 0;
                            }
                        }
                    }
                    if (__any_sync(0xffffffffu, found)) add |= (j < it.n0 ? 1u : 0u) | (j < it.n1 ? 2u : 0u);
                }
#pragma unroll 1
                for (int r = valid + sub; r < kKeys; r += kStep) *at(r) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->fixed[vat]);
            }
            g += 2 * n;
            // what was taken out of V goes to the rows that see it, once they are
            // stored (the next item's cannot be before this warp has cleared its tiles)
#pragma unroll 1
            for (int s = 0; s < 2; ++s) {
                if ((add >> s & 1u) && wait(&B->o_free[s], (stored >> s) & 1u)) {
                    const int first = it.tok0 + s * p.toks, end = min(first + p.toks, it.len);
#pragma unroll 1
                    for (int d = lane; d < HD; d += 32) {
                        const int plus = it.tok0 + M->since[0][d], minus = it.tok0 + M->since[1][d];
#pragma unroll 1
                        for (int tok = max(first, min(plus, minus)); tok < end; ++tok) {
                            const float inf = tok < plus ? -INFINITY : (tok < minus ? INFINITY : NAN);
                            uint16_t* x = p.out + ((size_t)(it.a + tok) * p.heads + (size_t)it.h * p.group) * HD + d;
#pragma unroll 1
                            for (int q = 0; q < p.group; ++q)
                                x[q * HD] = __bfloat16_as_ushort(__float2bfloat16_rn(bf16_bits_to_float(x[q * HD]) + inf));
                        }
                    }
                }
                if (it.n(s)) stored ^= 1u << s;
            }
        }
    }
}

// One time over the CTA's items: the softmax warps.
template <int HD, bool kSecond>
__device__ __forceinline__ void softmax_role(const Params& p, Misc* M, uint32_t tmem, int64_t total, int warp, int lane) {
    Bars* B = &M->b[kSecond];
    volatile WaitState* ab = &M->wst;
    Item it;

    // ---------------- softmax: thread = row
    const int s = (warp - 4) >> 2, wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lanes + (uint32_t)(s * 128);
    const uint32_t tO = tmem + lanes + (uint32_t)(256 + s * HD);
    const int rt = row / p.group, rg = row - rt * p.group;   // token and head of the row inside its tile
    const float c = p.scale2;
    const uint64_t c2 = pack2(c, c);
    uint32_t ns = 0, npv = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = __all_sync(0xffffffffu, wait_bar_here(bar, parity, ab));
        tc_fence_after();
        return ok;
    };
    for (int round = 0; ok && get_item(p, M, total, round, it); ++round) {
        const int n = it.n(s);
        if (!n) continue;
        const int tok = it.tok0 + s * p.toks + rt;           // sees keys 0 .. tok
        const int first = it.tok0 + s * p.toks;
        float ref = kFloorRef;
        uint64_t l2 = 0;                                     // two partial sums
        for (int j = 0; ok && j < n; ++j) {
            if (!wait(&B->s_full[s], ns++ & 1u)) break;
            float x[128];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32_async(tS + q * 32, x + q * 32);
            tmem_ready(x);
#pragma unroll
            for (int q = 1; q < 4; ++q) tmem_pin(x + q * 32);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B->s_read[s]);
            if ((j + 1) * kKeys - 1 > first) {               // a row of the tile does not see all keys
                const int lim = tok - j * kKeys;
                const float hidden = c < 0.f ? INFINITY : -INFINITY;
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    if (i > lim) x[i] = hidden;
            }
            // the row's largest score (a negative scale makes it the smallest product)
            float mx[4] = {x[0], x[1], x[2], x[3]};
            if (c >= 0.f) {
#pragma unroll
                for (int i = 4; i < 128; ++i) mx[i & 3] = fmaxf(mx[i & 3], x[i]);
            } else {
#pragma unroll
                for (int i = 4; i < 128; ++i) mx[i & 3] = fminf(mx[i & 3], x[i]);
            }
            const float top = c >= 0.f ? fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c
                                       : fminf(fminf(mx[0], mx[1]), fminf(mx[2], mx[3])) * c;
            if (__any_sync(0xffffffffu, top > ref + kLazy)) {
                // each row by its own scores alone: the others' do not reach its bits
                const float m = top > ref + kLazy ? top : ref, f = ex2_approx(ref - m);
                ref = m;
                float a, b;
                unpack2(l2, a, b);
                l2 = pack2(a * f, b * f);
                if (j > 0) {
                    if (!wait(&B->pv_done[s], (npv - 1u) & 1u)) break;
#pragma unroll
                    for (int q = 0; q < HD / 16; ++q) {
                        float o[16];
                        tmem_ldn<16>(tO + q * 16, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= f;
                        tmem_st16(tO + q * 16, o);
                    }
                }
            }
            const uint64_t r2 = pack2(-ref, -ref);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t pk[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float a, b;
                    unpack2(fma2(pack2(x[hf * 64 + 2 * i], x[hf * 64 + 2 * i + 1]), c2, r2), a, b);
                    a = ex2_approx(a);
                    b = ex2_approx(b);
                    l2 = add2(l2, pack2(a, b));
                    // bf16 for the product with V; the sum keeps float32
                    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                    pk[i] = reinterpret_cast<const uint32_t&>(h);
                }
                tmem_st32(tS + hf * 32, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->p_full[s][hf]);
            }
            ++npv;
        }
        if (!ok || !wait(&B->pv_done[s], (npv - 1u) & 1u)) break;
        float a, b;
        unpack2(l2, a, b);
        const float l = a + b, inv = 1.f / l;
        const bool valid = row < p.toks * p.group && tok < it.len;
        const size_t at = (size_t)(it.a + tok) * p.heads + (size_t)it.h * p.group + rg;
        uint32_t most = 0;                                   // bits of the row's largest magnitudes, a NaN's above all
#pragma unroll
        for (int q = 0; q < HD / 16; ++q) {
            float o[16];
            tmem_ldn<16>(tO + q * 16, o);
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
                pk[i] = reinterpret_cast<const uint32_t&>(h);
                most = __vmaxu2(most, pk[i] & 0x7FFF7FFFu);
            }
            if (valid) {
                uint4* dst = reinterpret_cast<uint4*>(p.out + at * HD + q * 16);
                dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B->o_free[s]);
        if (valid && p.lse) p.lse[at] = (ref + log2f(l)) * kLn2;
        if (__any_sync(0xffffffffu, valid && max(most & 0xFFFFu, most >> 16) >= 0x7F80u)) M->again = 1u;
    }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_kernel(const __grid_constant__ Maps maps, const Params p) {
    using C = Cfg<HD>;
    extern __shared__ uint8_t smem_raw[];
    // an offset, not an address rounded as an integer: the compiler keeps to
    // shared-memory instructions
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    Misc* M = reinterpret_cast<Misc*>(smem + C::kOffMisc);
    // by a shuffle: the compiler then knows that the warp's number, and what the
    // roles derive from it, is the same in every lane (12001 tokens 932 -> 796 us)
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        init_bars<HD>(&M->b[0]);
        M->wst.abort = 0;
        M->wst.limit = 1ull << 32;                            // until the workspace's own is read
        M->again = 0;
        prefetch_tmap(&maps.q);
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
    }
    if (warp == 1) tmem_alloc(&M->tmem, 512);
    // rows of Q that no token of an item fills are zeros (these for the whole
    // kernel, the rest item by item): their scores are 0 whatever ran before and
    // whatever the next sequence holds, so they never raise the references of
    // the rows beside them.
    for (int x = p.toks * p.group * 8 + threadIdx.x; x < kRows * 8; x += kThreads)
#pragma unroll
        for (int k = 0; k < 2 * C::kHalves; ++k)
            *reinterpret_cast<uint4*>(smem + C::kOffQ + k * C::kHalfBytes + x * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;                              // all 512 columns: they begin at the first
    // the kernel before this one: the list, or whatever the caller queued (the
    // workspace's header may be its work).  Waits read the limit anew each time
    // round, so no barrier follows.
    pdl_wait();
    if (threadIdx.x == 96) M->wst.limit = ws_wait_limit(p.ws);
    if (p.single) {
        if (blockIdx.x == 0) check_requests(p.seq_off, nullptr, p.B, p.T, 0, p.ws);
        if (warp == 2) {
            int64_t count;
            const int2 e = entry_of(p, blockIdx.x / p.kv_heads, count);
            if (lane == 0) {
                M->own = e;
                M->entries = (int)min(count, (int64_t)p.most);
            }
        }
        __syncthreads();
    }
    const int64_t total = (int64_t)__shfl_sync(0xffffffffu, p.single ? M->entries : __ldcg(p.count), 0) * p.kv_heads;
    // whether the CTA's items are gone over again, when all its warps are through
    // them (each warp asks once).  The second time is code of its own: one loop for
    // both took 922 us where this takes 788 (12001 tokens).
    auto again = [&]() {
        named_sync(1, kThreads);
        if (!__any_sync(0xffffffffu, M->again && !M->wst.abort)) return false;
        if (threadIdx.x == 0) init_bars<HD>(&M->b[1]);
        named_sync(1, kThreads);
        return true;
    };
    // registers: 384 x 168 at launch, then 128 x 104 + 256 x 200
    if (warp < 4) {
        regs_lower<104>();
        few_roles<HD, false>(maps, p, M, smem, tmem, total, warp, lane);
        if (again()) few_roles<HD, true>(maps, p, M, smem, tmem, total, warp, lane);
    } else {
        regs_raise<200>();
        softmax_role<HD, false>(p, M, tmem, total, warp, lane);
        if (again()) softmax_role<HD, true>(p, M, tmem, total, warp, lane);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && M->wst.abort) raise_status(p.ws, kStatTimeout);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int HD>
cudaError_t launch(const Maps& maps, const Params& p, cudaStream_t s) {
    const size_t smem = smem_bytes<HD>();
    cudaError_t e = allow_smem(attn_prompt_kernel<HD>, smem);
    if (e != cudaSuccess) return e;
    if (!p.single) {
        prof_begin(kPAttnPromptPlan, s);
        e = launch_kernel(attn_prompt_plan, dim3(1), dim3(kPlanThreads), 0, s, false, p, const_cast<int2*>(p.list),
                          const_cast<int*>(p.count));
        prof_end(s);
        if (e != cudaSuccess) return e;
    }
    prof_begin(kPAttnPrompt, s);
    e = launch_kernel(attn_prompt_kernel<HD>, dim3(num_sms()), dim3(kThreads), smem, s, true, maps, p);
    prof_end(s);
    return e;
}

int tile_tokens(int group) { return kRows / group; }

}  // namespace

// sum over sequences of ceil(tokens / pair) is at most T / pair + B
static size_t list_entries(int B, int T, int group) { return (size_t)T / (2 * tile_tokens(group)) + (size_t)B; }

size_t attn_prompt_workspace_bytes(int B, int T, int n_heads, int n_kv_heads, int) {
    return sizeof(WsHeader) + 256 + align_up(list_entries(B, T, n_heads / n_kv_heads) * sizeof(int2), 256);
}

cudaError_t launch_attn_prompt(const PromptArgs& a, cudaStream_t s) {
    uint8_t* w = static_cast<uint8_t*>(a.ws) + sizeof(WsHeader);
    Params p;
    p.seq_off = a.seq_off;
    p.count = reinterpret_cast<const int*>(w);
    p.list = reinterpret_cast<const int2*>(w + 256);
    p.out = static_cast<uint16_t*>(a.out);
    p.lse = a.lse;
    p.ws = a.ws;
    p.B = a.B;
    p.T = a.T;
    p.heads = a.n_heads;
    p.kv_heads = a.n_kv_heads;
    p.group = a.n_heads / a.n_kv_heads;
    p.toks = tile_tokens(p.group);
    p.most = (int)list_entries(a.B, a.T, p.group);
    // no CTA gets a second item: their order does not matter, so there is no
    // sort to wait for (8 sequences of 1 to 61 tokens, 4 key-value heads: 24 us
    // with the launch that sorts, 19 without)
    p.single = (int64_t)p.most * p.kv_heads <= num_sms();
    // hidden keys are infinite before the scale: at scale 0 the smallest normal
    // number keeps them so, and every finite score still counts as 0
    p.scale2 = a.scale == 0.f ? FLT_MIN : a.scale * kLog2e;
    Maps maps;
    auto map = [&](CUtensorMap* m, const void* base, int heads, int64_t stride, cuuint32_t b1, cuuint32_t b2) {
        const cuuint64_t dims[3] = {(cuuint64_t)a.head_dim, (cuuint64_t)heads, (cuuint64_t)a.T};
        const cuuint64_t str[2] = {(cuuint64_t)a.head_dim * 2, (cuuint64_t)stride * 2};
        const cuuint32_t box[3] = {64, b1, b2};
        return make_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if (!map(&maps.q, a.q, a.n_heads, a.q_stride, (cuuint32_t)p.group, (cuuint32_t)p.toks) ||
        !map(&maps.k, a.k, a.n_kv_heads, a.k_stride, 1, kKeys) || !map(&maps.v, a.v, a.n_kv_heads, a.v_stride, 1, kKeys))
        return cudaErrorInvalidValue;
    return a.head_dim == 64 ? launch<64>(maps, p, s) : launch<128>(maps, p, s);
}

}  // namespace dspark
