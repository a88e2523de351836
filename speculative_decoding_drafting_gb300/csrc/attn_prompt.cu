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
//   warp 3      zeroes the rows of a sequence's last V tile that are not its own
//               (0 times another sequence's NaN would be NaN), and sends
//               finished row tiles from their ring places to out
//   warps 4-11  softmax, one warpgroup per row tile, one row per thread: no
//               exchange between threads; the reference m is raised only when
//               a score exceeds it by more than 2^8, so the accumulator is
//               rescaled once or twice per item rather than at every tile.
//               Without a window the two take turns at their exponentials; with
//               one they work on half tiles (kSplit)
// Items (a pair of row tiles and a key-value head) are handed out from the
// longest to the shortest, forwards and backwards over the CTAs in turn.
//
// With a window (kWindow) an item's keys are the sinks and what its windows reach,
// one after another (Item): at most (head + window + tokens of the pair - 1) / 128 tiles,
// rounded up, wherever it stands.  With window 1024 a tile that every row sees takes 2550
// cycles, the two end tiles about 1000 more each, and the way to the next item 2700.
//
// 0 times a NaN or an infinity is NaN, so such a value in V would reach the rows
// that do not see its token too.  A CTA that has stored a row that is not finite goes
// over its items once more: warp 3 then takes what is not finite out of the V tiles
// that some row of the item does not see the whole of, and adds it to the rows
// that do see it when they are stored.  (Looking through those tiles in the
// first place made 12001 tokens 12 % and packed prompts 20 % slower: warp 3's
// loads wait behind the tensor core's reads of shared memory.)
//
// Bound by the tensor core and the softmax beside it: the two products of a
// tile of 128 x 128 scores take it about 1024 cycles at head_dim 128, and a turn
// of 128 exponentials a row as long.
// Measured (GB300): one sequence of 12001 tokens, 32 heads over 8 of 128: 740
// to 798 us, 1.48 to 1.60 PFLOP/s of the causal half (a plain bf16 product of
// 8192^3 runs at 1.91 in a burst and 1.70 under the power cap), of 64: 606 us; 16
// sequences of 100 to 4000 tokens: 504 to 553 us, 1.23 to 1.34 PFLOP/s.  30001 tokens,
// window 4096, 128 sinks: 1150 us by itself, 1243 to 1300 among other passes, 1.48 to 1.68;
// window 1024, 4 sinks: 412 to 425 us, 1.17 to 1.21; 16 sequences of 100 to 6000, window 1024:
// 600 to 650, 1.10 to 1.20.
// (Taking a quarter of the exponentials from the XU pipe to a polynomial on the FMA
// pipe cost 13 to 18 %: its instructions cost more than the pipe it relieves.)
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

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

// With a window a tile's 64 keys are a step of their own: their scores, weights and
// product follow one another while the other 64's do, in columns of their own, so that
// neither the tensor core nor the softmax waits for a whole tile of the other (30001
// tokens, window 4096, 1256 -> 1178 us; 16 of 100 to 6000, head_dim 64, window 1024, 520
// -> 464).  A row's reference then follows the halves.  Without one the reference
// follows whole tiles, which results' last bits depend on, and the row tiles take turns;
// turns of halves gained nothing.
template <bool kWindow>
constexpr bool kSplit = kWindow;

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
    // A row tile's result lies in its ring place: by place as well, since the softmax
    // may be through the next item's before warp 3 has looked at this one's.
    uint64_t staged[8];
    // A row tile's exponentials of a tile that both go over are made: the other's turn.
    uint64_t turn[2];
    uint64_t done;
    // kSplit: the scores of a tile's other 64 keys (s_full's are the first), and the
    // product with its first 64
    uint64_t s_more[2], pv_half[2];
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
    alignas(16) int4 own;
    int4 next[kThreads / 32];           // each warp's next entry of the list
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
    const int4* list;                   // pairs of row tiles (a sequence's first row, its tokens, the pair's first), longest first
    const int* count;                   // entries of the list
    int most;                           // entries that the workspace holds
    int single;                         // no CTA gets a second item: each finds its own entry
    int sectors;                        // out begins on a 32-byte boundary
    int bulk;                           // out is this device's memory: whole row tiles go there by bulk copies
    uint16_t* out;
    float* lse;
    void* ws;
    int B, T, heads, kv_heads, group, toks;   // toks: tokens of a row tile
    // with a window: its tokens, the first tokens that stay visible, and those in
    // whole copies; v as it lies in memory (for values that are not finite)
    int window, sinks, head;
    const uint16_t* v;
    int64_t v_stride;
    float scale2;                       // |scale| log2(e)
    int negate;                         // a negative scale: the products are negated
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
__global__ void __launch_bounds__(kPlanThreads) attn_prompt_plan(Params p, int4* list, int* count) {
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
            for (int t = lane; t < n; t += 32) f(r, t, kPlanThreads - 1 - (int)((int64_t)t * kPlanThreads / n_class));
        }
    };
    each([&](const RowRange&, int, int c) { atomicAdd(&at[c], u64(1)); });
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
    each([&](const RowRange& r, int t, int c) {
        const u64 k = atomicAdd(&at[c], u64(1));
        if (k < (u64)p.most) list[k] = make_int4(r.a, r.b - r.a, t * pair, 0);
    });
}

// With a window an item's keys are the sinks (rounded up to kHeadRows, `head`) and
// those from the first that row tile 0's first window holds up to its end, one
// after another; its tiles are cut from that line, in which place v stands for key
// v, or v + gap from the head's end on.  (Tiles of the keys themselves took one for
// the sinks alone and half of one before the window: 10 for a window of 1024 and 4
// sinks where this takes 9, with four query heads to a key-value head.)  Where nothing is
// left out, head and gap are 0.
constexpr int kHeadRows = 8;            // rows of a swizzle atom, which a copy can fill by itself
template <bool kWindow>
struct Item {
    int a, len;                         // the sequence's first row and its tokens
    int tok0;                           // first token of row tile 0
    int h;                              // key-value head
    int n0, n1;                         // key tiles up to each row tile's last (0: no rows)
    int keys;                           // keys that the item's last token sees
    int head, gap, lead;                // with a window; lead: tiles that row tile 1 sees nothing of
    __device__ __forceinline__ int n(int s) const { return s ? n1 : n0; }
    __device__ __forceinline__ int tiles() const { return max(n0, n1); }
    // Places of the ring that the item takes: K and V of its tiles, and the first time
    // one for each row tile's result (the tiles are equally large).
    __device__ __forceinline__ int results(bool second) const { return second ? 0 : (n1 ? 2 : 1); }
    __device__ __forceinline__ uint32_t places(bool second) const { return (uint32_t)(2 * tiles() + results(second)); }
    // row tile s goes over tiles begin(s) to n(s)
    __device__ __forceinline__ int begin(int s) const { return kWindow && s && n1 ? lead : 0; }
    __device__ __forceinline__ int key(int v) const { return kWindow && v >= head ? v + gap : v; }
    // what tile j's first row would stand for as a key if its last row's key decides
    __device__ __forceinline__ int key0(int j) const { return key(j * kKeys + kKeys - 1) - (kKeys - 1); }
    // V tiles to clear: from this one on, those with rows past the sequence's end, or,
    // the second time, with a key that some row of the item does not see.  (The
    // first time with rows past the item's keys, later tokens of the sequence: their
    // weights are 0, and if one is not finite the second time comes anyway; to clear
    // them took window 1024 packed 630 us for 609.)
    __device__ __forceinline__ int edge(bool second) const {
        return second ? min((tok0 + 1 - gap) / kKeys, tiles() - 1) : (tiles() * kKeys + gap <= len ? tiles() : (keys - gap) / kKeys);
    }
    // (with a window, the second time, also some of those before)
    __device__ __forceinline__ bool clears(const Params& p, int j, bool second) const {
        return j >= edge(second) || (kWindow && second && key0(j) < keys - p.window && (j + 1) * kKeys > p.sinks);
    }
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

// A CTA's items in turn, asked for by whole warps.  The list's entry for the next one
// is on its way to the warp's place in shared memory while this one is worked on:
// items with a window are short, and a load from L2 before each took 5 to 20 % of
// them.  (Kept in registers it slowed the softmax's loop by 10 %.)
template <bool kWindow>
__device__ __forceinline__ bool get_item(const Params& p, Misc* M, int64_t total, int round, Item<kWindow>& it) {
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
    const uint64_t n = gridDim.x, c = blockIdx.x;
    auto place = [&](int r) { return (uint64_t)r * n + ((r & 1) ? n - 1 - c : c); };
    auto entry = [&](uint64_t k) { return (uint64_t)total >> 32 ? k / (uint32_t)p.kv_heads : (uint32_t)k / (uint32_t)p.kv_heads; };
    // the list was written by the kernel before this one
    auto ask = [&](uint64_t k) {
        if (elect_one()) cp_async16_zf(&M->next[warp], p.list + entry(k), 16u);
    };
    const uint64_t k = place(round);
    if (k >= (uint64_t)total) return false;
    int4 e;
    if (p.single) {
        e = M->own;
    } else {
        if (round == 0) ask(k);
        cp_async_wait_all();
        __syncwarp();
        e = M->next[warp];
        __syncwarp();
        if (place(round + 1) < (uint64_t)total) ask(place(round + 1));
    }
    it.h = (int)(k - entry(k) * (uint32_t)p.kv_heads);
    it.a = __shfl_sync(0xffffffffu, e.x, 0);                  // the same in every lane, as the compiler now knows
    it.len = __shfl_sync(0xffffffffu, e.y, 0);
    it.tok0 = __shfl_sync(0xffffffffu, e.z, 0);
    it.head = it.gap = it.lead = 0;
    if (kWindow) {
        const int low = it.tok0 - p.window + 1;
        if (low > p.head) {
            it.head = p.head;
            it.gap = low - p.head;
            it.lead = p.head ? 0 : p.toks / kKeys;
        }
    }
    auto tiles = [&](int first) {
        return first < it.len ? (min(it.len, first + p.toks) - it.gap + kKeys - 1) / kKeys : 0;
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

// 32 bytes; at once where `sectors` says that they begin on a 32-byte boundary.
__device__ __forceinline__ void store32(uint16_t* dst, const uint32_t (&v)[8], bool sectors) {
    if (sectors) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

struct Maps {
    CUtensorMap q, k, v;
    CUtensorMap k_head, v_head;         // with a window: kHeadRows rows
    CUtensorMap out;
};

template <int HD>
__device__ __forceinline__ void init_bars(Bars* B) {
    using C = Cfg<HD>;
    for (int i = 0; i < C::kStages; ++i) {
        mbar_init(&B->full[i], 1);
        mbar_init(&B->empty[i], 2);
        mbar_init(&B->fixed[i], 1);
        mbar_init(&B->staged[i], 4);
    }
    for (int s = 0; s < 2; ++s) {
        mbar_init(&B->q_full[s], 1);
        mbar_init(&B->q_empty[s], 1);
        mbar_init(&B->s_full[s], 1);
        mbar_init(&B->s_more[s], 1);
        mbar_init(&B->s_read[s], 4);
        mbar_init(&B->p_full[s][0], 4);
        mbar_init(&B->p_full[s][1], 4);
        mbar_init(&B->asked[s], 1);
        mbar_init(&B->turn[s], 4);
        mbar_init(&B->pv_half[s], 1);
        mbar_init(&B->pv_done[s], 1);
        mbar_init(&B->o_free[s], 4);
    }
    mbar_init(&B->done, 2);
    fence_mbar_init();
}

// One time over the CTA's items: warps 0 to 3.
template <int HD, bool kWindow, bool kSecond>
__device__ __forceinline__ void few_roles(const Maps& maps, const Params& p, Misc* M, uint8_t* smem, uint32_t tmem,
                                          int64_t total, int warp, int lane) {
    using C = Cfg<HD>;
    Bars* B = &M->b[kSecond];
    volatile WaitState* ab = &M->wst;
    Item<kWindow> it = {};

    if (warp == 0) {
        // ---------------- producer
        const uint64_t pol_q = policy_evict_first(), pol_kv = policy_evict_last();
        uint32_t g = 0, st = 0, ph = 0, nq = 0, used = 0;     // tiles issued; the next ring place and its phase; Q's
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, wait_bar_here(bar, parity, ab)); };
        auto tile = [&](const CUtensorMap* m, const CUtensorMap* head, int j) {
            wait(&B->empty[st], ph ^ 1u);
            if (!ok) return;
            if (kWindow && j * kKeys < it.head && (j + 1) * kKeys > it.head) {
                // the end of the sinks and the beginning of the window, 8 rows to a copy
                if (elect_one()) mbar_expect_tx(&B->full[st], (uint32_t)C::kTileBytes);
                __syncwarp();
                if (lane < kKeys / kHeadRows) {
#pragma unroll
                    for (int hf = 0; hf < C::kHalves; ++hf)
                        tma_load_3d(smem + st * C::kTileBytes + hf * C::kHalfBytes + lane * (kHeadRows * 128), head, &B->full[st],
                                    hf * 64, it.h, it.a + it.key(j * kKeys + lane * kHeadRows), pol_kv);
                }
            } else if (elect_one()) {
                mbar_expect_tx(&B->full[st], (uint32_t)C::kTileBytes);
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf)
                    tma_load_3d(smem + st * C::kTileBytes + hf * C::kHalfBytes, m, &B->full[st], hf * 64, it.h,
                                it.a + it.key(j * kKeys), pol_kv);
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
            tile(&maps.k, &maps.k_head, 0);
            query(1);
#pragma unroll 1
            for (int j = 0; ok && j < n; ++j) {
                if (j) tile(&maps.k, &maps.k_head, j);
                tile(&maps.v, &maps.v_head, j);
            }
            // places for the results
#pragma unroll 1
            for (int s = 0; ok && s < it.results(kSecond); ++s) {
                wait(&B->empty[st], ph ^ 1u);
                if (!ok) break;
                if (lane == 0) mbar_arrive(&B->full[st]);
                __syncwarp();
                ++g;
                if (++st == C::kStages) {
                    st = 0;
                    ph ^= 1u;
                }
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
        // (a negative scale: bit 13 negates Q)
        const uint32_t id_qk = idesc_bf16_f32(128, 64, false, false) | (uint32_t)p.negate << 13;
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
                if (kSplit<kWindow> || !half) umma_commit(kSplit<kWindow> && half ? &B->s_more[s] : &B->s_full[s]);
                if (kSplit<kWindow> ? half : !half) {
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
            const int j0 = it.begin(s);
            // tiles that only the other row tile sees, before this one's
#pragma unroll 1
            for (int j = 0; kWindow && ok && j < 2 * j0; ++j) {
                if (!wait(&B->full[st], ph)) break;
                if (lane == 0) mbar_arrive(&B->empty[st]);
                if ((j & 1) && it.clears(p, j >> 1, kSecond)) nfix ^= 1u << st;
                next();
            }
            if (!wait(&B->full[st], ph)) break;
            if (it.n(s)) {
                // (the item before it has been read and multiplied)
                scores(st, kSplit<kWindow> ? 0 : 1, j0);
                scores(st, kSplit<kWindow> ? 1 : 0, j0);
            } else if (lane == 0) {
                mbar_arrive(&B->empty[st]);
            }
            next();
#pragma unroll 1
            for (int j = j0; ok && j < n; ++j) {
                // V_j at st, K_{j+1} at the place after it
                const uint32_t vat = st, vph = ph;
                next();
                const uint32_t kat = st, kph = ph;
                if (j + 1 < n) next();
                if (!kSplit<kWindow> && j < it.n(s)) {
                    if (!wait(&B->s_read[s], nr & 1u)) break;
                    nr ^= 1u;
                    if (j + 1 < it.n(s)) {
                        if (!wait(&B->full[kat], kph)) break;
                        scores(kat, 1, j + 1);
                    }
                }
                if (!wait(&B->full[vat], vph)) break;
                const bool fix = it.clears(p, j, kSecond);
                if (j < it.n(s)) {
                    // warp 3 starts while P is still being made
                    if (fix && lane == 0) mbar_arrive(&B->asked[s]);
                    if (j == j0) {
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
                                umma_bf16_ts(tO, tS + half * (kSplit<kWindow> ? 64 : 32) + kk * 8, b + kk * 128, id_pv,
                                             ((j - j0) | half | kk) ? 1u : 0u);
                            if (kSplit<kWindow> && !half) umma_commit(&B->pv_half[s]);
                            if (half) {
                                umma_commit(&B->pv_done[s]);
                                umma_commit(&B->empty[vat]);
                            }
                        }
                        __syncwarp();
                        if (kSplit<kWindow> && j + 1 < it.n(s)) {
                            if (!half && !wait(&B->full[kat], kph)) break;
                            scores(kat, half, j + 1);
                        }
                    }
                    if (!ok) break;
                    np ^= 1u;
                    if (!kSplit<kWindow> && j + 1 < it.n(s)) scores(kat, 0, j + 1);
                } else if (lane == 0) {
                    mbar_arrive(&B->empty[vat]);
                }
                if (fix) nfix ^= 1u << vat;
                if (j + 1 < n && j + 1 >= it.n(s)) {          // a tile only the other row tile sees
                    if (!wait(&B->full[kat], kph)) break;
                    if (lane == 0) mbar_arrive(&B->empty[kat]);
                }
            }
#pragma unroll 1
            for (int i = 0; i < it.results(kSecond); ++i) next();
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
        uint32_t asked = 0;                                   // parity of each row tile's next request, by bit
        [[maybe_unused]] uint32_t stored = 0;                 // the second time: and of its next item's stores
        uint32_t laid = 0;                                    // of each ring place's next result
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
            for (int j = kWindow && kSecond ? 0 : it.edge(kSecond); j < n; ++j) {
                if (kWindow && kSecond && !it.clears(p, j, kSecond)) continue;
                const int key0 = it.key0(j);
                // the issuers that use the tile have seen it arrive (its parity alone
                // could be an earlier tile's)
                const uint32_t vi = g + 2 * j + 1, vat = vi % C::kStages;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (j < it.begin(s) || j >= it.n(s)) continue;
                    wait(&B->asked[s], (asked >> s) & 1u);
                    asked ^= 1u << s;
                }
                if (!wait(&B->full[vat], (vi / C::kStages) & 1u)) break;
                uint8_t* vt = smem + vat * C::kTileBytes + (piece / 8) * C::kHalfBytes;
                auto at = [&](int row) { return reinterpret_cast<uint4*>(vt + row * 128 + ((piece ^ row) & 7) * 16); };
                const int valid = min(it.keys - key0, kKeys);
                if (kSecond && kWindow) {
                    // whatever is not finite goes; which rows see it is worked out below
                    bool found = false;
#pragma unroll 1
                    for (int row = sub; row < valid; row += kStep) {
                        uint4 w = *at(row);
                        uint32_t x[4] = {w.x, w.y, w.z, w.w};
                        bool bad = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t m = x[e] & 0x7FFF7FFFu;
                            if ((m & 0xFFFFu) >= 0x7F80u) x[e] &= 0xFFFF0000u, bad = true;
                            if (m >= 0x7F800000u) x[e] &= 0xFFFFu, bad = true;
                        }
                        if (bad) *at(row) = make_uint4(x[0], x[1], x[2], x[3]);
                        found |= bad;
                    }
                    if (__any_sync(0xffffffffu, found))
                        add |= (it.begin(0) <= j && j < it.n0 ? 1u : 0u) | (it.begin(1) <= j && j < it.n1 ? 2u : 0u);
                } else if (kSecond) {
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
            // the results go from their ring places to out, but for those of a sequence's end
#pragma unroll 1
            for (int s = 0; s < it.results(kSecond); ++s) {
                const uint32_t at = (g + 2 * n + s) % C::kStages;
                if (!wait(&B->staged[at], (laid >> at) & 1u)) break;
                laid ^= 1u << at;
                if (lane == 0) {
                    const int first = it.tok0 + s * p.toks;
                    if (p.bulk && first + p.toks <= it.len) {
#pragma unroll
                        for (int hf = 0; hf < C::kHalves; ++hf)
                            tma_store_3d(&maps.out, smem + at * C::kTileBytes + hf * C::kHalfBytes, hf * 64, it.h * p.group, it.a + first);
                        tma_store_commit();
                        tma_store_wait_read();
                    }
                    mbar_arrive(&B->empty[at]);
                    mbar_arrive(&B->empty[at]);
                }
                __syncwarp();
            }
            g += it.places(kSecond);
            // What was taken out of V goes to the rows that see it, once they are
            // stored.  The stores of items with nothing to add are waited for too, so that
            // this warp's count of them is never behind: with a window the issuers ask
            // for an item's tiles before the one before it is stored, and a wait for this
            // item's parity alone would then pass at once, and the softmax store over
            // what was added.  (Nor can stores run ahead: a row tile has a tile to be
            // cleared in each of its items.)
#pragma unroll 1
            for (int s = 0; kSecond && s < 2; ++s) {
                if (!it.n(s)) continue;
                if (!wait(&B->o_free[s], (stored >> s) & 1u)) break;
                stored ^= 1u << s;
                if (add >> s & 1u) {
                    const int first = it.tok0 + s * p.toks, end = min(first + p.toks, it.len);
                    if constexpr (kWindow) {
                        // the cleared tiles' keys in their order, each when the first token
                        // that sees it comes: the latest that holds an infinity (a NaN
                        // counts as both) and the first among the sinks decide a token
#pragma unroll 1
                        for (int d = lane; d < HD; d += 32) {
                            const uint16_t* v = p.v + (int64_t)it.a * p.v_stride + (int64_t)it.h * HD + d;
                            int plus = -1, minus = -1, plus_sink = 0x7FFFFFFF, minus_sink = 0x7FFFFFFF, at = 0;
#pragma unroll 1
                            for (int tok = first; tok < end; ++tok) {
#pragma unroll 1
                                while (at < n * kKeys) {
                                    const int k = it.key(at);
                                    if (k > tok) break;
                                    if (!it.clears(p, at / kKeys, true)) {
                                        at = (at / kKeys + 1) * kKeys;
                                        continue;
                                    }
                                    const bool none = at >= p.sinks && at < it.head;      // between the sinks and the head's end
                                    ++at;
                                    if (none) continue;
                                    const uint32_t x = v[(int64_t)k * p.v_stride];
                                    if ((x & 0x7F80u) != 0x7F80u) continue;
                                    if ((x & 0x7Fu) || !(x & 0x8000u)) {
                                        plus = k;
                                        if (k < p.sinks) plus_sink = min(plus_sink, k);
                                    }
                                    if ((x & 0x7Fu) || (x & 0x8000u)) {
                                        minus = k;
                                        if (k < p.sinks) minus_sink = min(minus_sink, k);
                                    }
                                }
                                const int low = tok - p.window;
                                const bool up = (plus >= 0 && plus > low) || plus_sink <= tok;
                                const bool down = (minus >= 0 && minus > low) || minus_sink <= tok;
                                if (!up && !down) continue;
                                const float inf = up ? (down ? NAN : INFINITY) : -INFINITY;
                                uint16_t* x = p.out + ((size_t)(it.a + tok) * p.heads + (size_t)it.h * p.group) * HD + d;
#pragma unroll 1
                                for (int q = 0; q < p.group; ++q)
                                    x[q * HD] = __bfloat16_as_ushort(__float2bfloat16_rn(bf16_bits_to_float(x[q * HD]) + inf));
                            }
                        }
                    } else {
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
                }
            }
        }
        // what the second time stores comes after
        if (!kSecond) {
            if (lane == 0) tma_store_wait();
            __syncwarp();
        }
    }
}

// One time over the CTA's items: the softmax warps.
template <int HD, bool kWindow, bool kSecond>
__device__ __forceinline__ void softmax_role(const Params& p, Misc* M, uint8_t* smem, uint32_t tmem, int64_t total, int warp, int lane) {
    using C = Cfg<HD>;
    Bars* B = &M->b[kSecond];
    volatile WaitState* ab = &M->wst;
    Item<kWindow> it = {};

    // ---------------- softmax: thread = row
    const int s = (warp - 4) >> 2, wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lanes + (uint32_t)(s * 128);
    const uint32_t tO = tmem + lanes + (uint32_t)(256 + s * HD);
    const int rt = row / p.group, rg = row - rt * p.group;   // token and head of the row inside its tile
    const float c = p.scale2;
    const uint64_t c2 = pack2(c, c);
    uint32_t ns = 0, npv = 0, g = 0;                         // g: ring places before this item
    // Without a window the two row tiles take turns at the exponentials of the tiles that both go over,
    // row tile 0 first, so that one's run beside the other's products.  Left alone they
    // settled in step or out of step as small changes of the code would have it: both
    // at the exponentials at once, 12001 tokens took 893 us, out of step 780, and in
    // turns they take 730 (head_dim 64: 693, 661, 610).
    uint32_t nt = 0;                                         // such tiles so far
    auto in_turns = [&](int j) { return j < min(it.n0, it.n1); };
    auto hand_over = [&](int j) {
        if (in_turns(j) && lane == 0) mbar_arrive(&B->turn[1 - s]);
    };
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = __all_sync(0xffffffffu, wait_bar_here(bar, parity, ab));
        tc_fence_after();
        return ok;
    };
    // (with a window, whose items are short, the next one is worked out while the last
    // product of this one runs: window 128 187 -> 160 us, window 1024 packed 612 -> 597)
    Item<kWindow> coming = {};
    bool more = kWindow && get_item(p, M, total, 0, coming);
    for (int round = 0; ok && (kWindow ? more : get_item(p, M, total, round, it)); ++round) {
        if (kWindow) it = coming;
        const int n = it.n(s), j0 = it.begin(s);
        const uint32_t mine = g + (uint32_t)(2 * it.tiles() + s);   // the ring place for the result
        g += it.places(kSecond);
        if (!n) {
            if (kWindow) more = get_item(p, M, total, round + 1, coming);
            continue;
        }
        const int tok = it.tok0 + s * p.toks + rt;           // sees keys 0 .. tok
        const int first = it.tok0 + s * p.toks;
        float ref = kFloorRef;
        uint64_t l2 = 0;                                     // two partial sums
        // 64 keys of tile j
        auto half_tile = [&](int j, int hf, auto masked) {
            if (!wait(hf ? &B->s_more[s] : &B->s_full[s], ns & 1u)) return false;
            float x[64];
            tmem_ld32_async(tS + hf * 64, x);
            tmem_ld32_async(tS + hf * 64 + 32, x + 32);
            tmem_ready(x);
            tmem_pin(x + 32);
            if constexpr (decltype(masked)::value) {
                // neither the keys behind it nor, but for the sinks, those before its window
                const int key0 = it.key0(j) + hf * 64, sees = tok - key0 + 1, low = sees - p.window, sink = p.sinks - j * kKeys - hf * 64;
                auto first_bits = [](int n) { return n <= 0 ? 0u : 0xFFFFFFFFu >> (32 - min(n, 32)); };
#pragma unroll
                for (int q = 0; q < 64; q += 32) {
                    const uint32_t seen = first_bits(sees - q) & (~first_bits(low - q) | first_bits(sink - q));
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!((seen >> i) & 1u)) x[q + i] = -INFINITY;
                }
            }
            // the row's largest score
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int i = 4; i < 64; ++i) mx[i & 3] = fmaxf(mx[i & 3], x[i]);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
            if (__any_sync(0xffffffffu, top > ref + kLazy)) {
                // each row by its own scores alone: the others' do not reach its bits
                const float m = top > ref + kLazy ? top : ref, f = ex2_approx(ref - m);
                ref = m;
                float a, b;
                unpack2(l2, a, b);
                l2 = pack2(a * f, b * f);
                if (j > j0 || hf) {                          // what the accumulator holds so far
                    if (!wait(hf ? &B->pv_half[s] : &B->pv_done[s], (hf ? npv : npv - 1u) & 1u)) return false;
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
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                float a, b;
                unpack2(fma2(pack2(x[2 * i], x[2 * i + 1]), c2, r2), a, b);
                a = ex2_approx(a);
                b = ex2_approx(b);
                l2 = add2(l2, pack2(a, b));
                // bf16 for the product with V (half a step: 2^-9 of the binade), whose factors
                // the tensor core takes at that rate; the sum keeps float32
                const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                pk[i] = reinterpret_cast<const uint32_t&>(h);
            }
            tmem_st32(tS + hf * 64, pk);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B->p_full[s][hf]);
            return true;
        };
        auto tile = [&](int j, [[maybe_unused]] auto masked) {
            if constexpr (kSplit<kWindow>) {
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf)
                    if (!half_tile(j, hf, masked)) return false;
                ++ns;
                ++npv;
                return true;
            }
            if (!wait(&B->s_full[s], ns++ & 1u)) return false;
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
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    if (i > lim) x[i] = -INFINITY;
            }
            // the row's largest score
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int i = 4; i < 128; ++i) mx[i & 3] = fmaxf(mx[i & 3], x[i]);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
            if (__any_sync(0xffffffffu, top > ref + kLazy)) {
                // each row by its own scores alone: the others' do not reach its bits
                const float m = top > ref + kLazy ? top : ref, f = ex2_approx(ref - m);
                ref = m;
                float a, b;
                unpack2(l2, a, b);
                l2 = pack2(a * f, b * f);
                if (j > j0) {
                    if (!wait(&B->pv_done[s], (npv - 1u) & 1u)) return false;
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
            if (in_turns(j)) {
                if ((s || nt) && !wait(&B->turn[s], (s ? nt : nt - 1u) & 1u)) return false;
                ++nt;
            }
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
                    // bf16 for the product with V, as above; the sum keeps float32
                    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                    pk[i] = reinterpret_cast<const uint32_t&>(h);
                }
                tmem_st32(tS + hf * 32, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->p_full[s][hf]);
                if (hf) hand_over(j);
            }
            ++npv;
            return true;
        };
        if constexpr (kWindow) {
            // Whole sinks' tiles, those that some window begins in or behind, whole ones,
            // the diagonal's: with the tests in one loop for all (in registers, or as
            // a pass over the scores in tensor memory) the whole ones took 15 % longer.
            const int full = max((first + 1 - it.gap) / kKeys, 0);                          // from here on: the diagonal
            const int clean[2] = {min(min(p.sinks / kKeys, full), n), min(full, n)};
            const int ends[2] = {min(max((first + p.toks - p.window - it.gap + kKeys - 1) / kKeys, 0), n), n};
            int j = j0;
#pragma unroll 1
            for (int part = 0; ok && part < 2; ++part) {
#pragma unroll 1
                for (const int to = part ? clean[1] : clean[0]; ok && j < to; ++j)
                    if (!tile(j, std::false_type{})) break;
#pragma unroll 1
                for (const int to = part ? ends[1] : ends[0]; ok && j < to; ++j)
                    if (!tile(j, std::true_type{})) break;
            }
        } else {
            for (int j = 0; ok && j < n; ++j)
                if (!tile(j, std::false_type{})) break;
        }
        if (!ok) break;
        const bool valid = row < p.toks * p.group && tok < it.len;
        const size_t at = (size_t)(it.a + tok) * p.heads + (size_t)it.h * p.group + rg;
        const bool direct = kSecond || !p.bulk || first + p.toks > it.len;
        if (kWindow) more = get_item(p, M, total, round + 1, coming);
        if (!wait(&B->pv_done[s], (npv - 1u) & 1u)) break;
        float a, b;
        unpack2(l2, a, b);
        const float l = a + b, inv = 1.f / l;
        // the accumulator is read at once and free for the next item before its rows
        // are stored (but warp 3 mends stored rows)
        float o[HD];
#pragma unroll
        for (int q = 0; q < HD / 32; ++q) tmem_ld32_async(tO + q * 32, o + q * 32);
        tmem_ready(o);
#pragma unroll
        for (int q = 1; q < HD / 32; ++q) tmem_pin(o + q * 32);
        tc_fence_before();
        if (!kSecond) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&B->o_free[s]);
        }
        // A whole row tile goes to out by way of a ring place: rows lie 32 to an
        // instruction, one per lane, and stored as they are took 5000 cycles of the 16000
        // to 40000 of an item.  The last one of a sequence must not touch the rows
        // behind it; what is mended is stored as it is, and so is an out that is not this
        // device's memory (mapped host memory, a peer's): plain stores reach any of them.
        uint8_t* stage = smem + mine % C::kStages * C::kTileBytes;
        if (!kSecond && !wait(&B->full[mine % C::kStages], mine / C::kStages & 1u)) break;
        uint32_t most = 0;                                   // bits of the row's largest magnitudes, a NaN's above all
#pragma unroll
        for (int q = 0; q < HD / 16; ++q) {
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(o[q * 16 + 2 * i] * inv, o[q * 16 + 2 * i + 1] * inv);
                pk[i] = reinterpret_cast<const uint32_t&>(h);
                most = __vmaxu2(most, pk[i] & 0x7FFF7FFFu);
            }
            if (!direct) {
                uint8_t* to = stage + (q / 4) * C::kHalfBytes + row * 128;
                const int c0 = q % 4 * 2;
                *reinterpret_cast<uint4*>(to + ((c0 ^ row) & 7) * 16) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                *reinterpret_cast<uint4*>(to + (((c0 + 1) ^ row) & 7) * 16) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
            } else if (valid) {
                // a whole sector per lane and store, where out allows it
                store32(p.out + at * HD + q * 16, pk, p.sectors);
            }
        }
        if (!kSecond) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B->staged[mine % C::kStages]);
        }
        if (kSecond) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&B->o_free[s]);
        }
        if (valid && p.lse) p.lse[at] = (ref + log2f(l)) * kLn2;
        if (__any_sync(0xffffffffu, valid && max(most & 0xFFFFu, most >> 16) >= 0x7F80u)) M->again = 1u;
    }
}

template <int HD, bool kWindow>
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
        if (p.bulk) prefetch_tmap(&maps.out);
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
                const RowRange r = row_range(p.seq_off, e.x, p.T);
                M->own = make_int4(r.a, r.b - r.a, e.y * 2 * p.toks, 0);
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
        few_roles<HD, kWindow, false>(maps, p, M, smem, tmem, total, warp, lane);
        if (again()) few_roles<HD, kWindow, true>(maps, p, M, smem, tmem, total, warp, lane);
    } else {
        regs_raise<200>();
        softmax_role<HD, kWindow, false>(p, M, smem, tmem, total, warp, lane);
        if (again()) softmax_role<HD, kWindow, true>(p, M, smem, tmem, total, warp, lane);
    }
    cp_async_wait_all();                                      // an entry asked for before a wait ran out
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && M->wst.abort) raise_status(p.ws, kStatTimeout);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int HD, bool kWindow>
cudaError_t launch(const Maps& maps, const Params& p, cudaStream_t s) {
    const size_t smem = smem_bytes<HD>();
    cudaError_t e = allow_smem(attn_prompt_kernel<HD, kWindow>, smem);
    if (e != cudaSuccess) return e;
    if (!p.single) {
        prof_begin(kPAttnPromptPlan, s);
        e = launch_kernel(attn_prompt_plan, dim3(1), dim3(kPlanThreads), 0, s, false, p, const_cast<int4*>(p.list),
                          const_cast<int*>(p.count));
        prof_end(s);
        if (e != cudaSuccess) return e;
    }
    prof_begin(kPAttnPrompt, s);
    e = launch_kernel(attn_prompt_kernel<HD, kWindow>, dim3(num_sms()), dim3(kThreads), smem, s, true, maps, p);
    prof_end(s);
    return e;
}

int tile_tokens(int group) { return kRows / group; }

}  // namespace

// sum over sequences of ceil(tokens / pair) is at most T / pair + B
static size_t list_entries(int B, int T, int group) { return (size_t)T / (2 * tile_tokens(group)) + (size_t)B; }

size_t attn_prompt_workspace_bytes(int B, int T, int n_heads, int n_kv_heads, int) {
    return sizeof(WsHeader) + 256 + align_up(list_entries(B, T, n_heads / n_kv_heads) * sizeof(int4), 256);
}

cudaError_t launch_attn_prompt(const PromptArgs& a, cudaStream_t s) {
    uint8_t* w = static_cast<uint8_t*>(a.ws) + sizeof(WsHeader);
    Params p = {};
    p.seq_off = a.seq_off;
    p.count = reinterpret_cast<const int*>(w);
    p.list = reinterpret_cast<const int4*>(w + 256);
    p.out = static_cast<uint16_t*>(a.out);
    p.sectors = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    p.bulk = a.out_on_device;
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
    p.scale2 = a.scale == 0.f ? FLT_MIN : std::fabs(a.scale) * kLog2e;
    p.negate = a.scale < 0.f;
    Maps maps = {};
    auto map = [&](CUtensorMap* m, const void* base, int heads, int64_t stride, cuuint32_t b1, cuuint32_t b2) {
        const cuuint64_t dims[3] = {(cuuint64_t)a.head_dim, (cuuint64_t)heads, (cuuint64_t)a.T};
        const cuuint64_t str[2] = {(cuuint64_t)a.head_dim * 2, (cuuint64_t)stride * 2};
        const cuuint32_t box[3] = {64, b1, b2};
        return make_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if (p.bulk && !map(&maps.out, a.out, a.n_heads, (int64_t)a.n_heads * a.head_dim, (cuuint32_t)p.group, (cuuint32_t)p.toks)) return cudaErrorInvalidValue;
    if (!map(&maps.q, a.q, a.n_heads, a.q_stride, (cuuint32_t)p.group, (cuuint32_t)p.toks) ||
        !map(&maps.k, a.k, a.n_kv_heads, a.k_stride, 1, kKeys) || !map(&maps.v, a.v, a.n_kv_heads, a.v_stride, 1, kKeys))
        return cudaErrorInvalidValue;
    // a window of every token is none
    if (a.window > 0 && a.window < a.T) {
        p.window = a.window;
        p.sinks = a.sinks < a.T ? a.sinks : a.T;
        p.head = (int)std::min(((int64_t)p.sinks + kHeadRows - 1) / kHeadRows * kHeadRows, (int64_t)0x7FFFFFFF);
        if (!map(&maps.k_head, a.k, a.n_kv_heads, a.k_stride, 1, kHeadRows) ||
            !map(&maps.v_head, a.v, a.n_kv_heads, a.v_stride, 1, kHeadRows))
            return cudaErrorInvalidValue;
        p.v = static_cast<const uint16_t*>(a.v);
        p.v_stride = a.v_stride;
        return a.head_dim == 64 ? launch<64, true>(maps, p, s) : launch<128, true>(maps, p, s);
    }
    return a.head_dim == 64 ? launch<64, false>(maps, p, s) : launch<128, false>(maps, p, s);
}

}  // namespace dspark
