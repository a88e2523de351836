// attn_plan.h -- how paged attention splits its work (plain C++, also
// compiled for the host, where its index ranges are checked).
//
// An item is one row tile of one request and one key-value head: up to
// kRowTile of the request's rows (row = new token x query heads of the group,
// heads fastest) over the keys that its last row sees, in tiles of kKeyTile
// keys, at least one.  Items are numbered request, row tile, head and laid one
// after another on a line, each as long as it is expected to take: `start` and
// a length per key tile that depends on its rows.  The line is cut into equal
// spans, one per CTA, and a CTA takes the key tiles that begin in its span, so
// that requests of any mix of lengths load the device evenly.  An item that a
// cut goes through leaves one partial result per piece.
//
// With a window (WindowPlan) an item's keys are the sinks' pages and, from the
// page that its first row's window begins in, those up to its end, one after
// another; its tiles are cut from that line, in which key v stands for key v, or
// v + gap from the sinks' end on.  One token's line is at most
// head + window + unit - 1 long (WindowPlan).  (Tiles of the keys themselves left a
// tile to the sinks and one to the window's beginning, mostly hidden: 10 tiles for
// a window of 1024 and 4 sinks where this takes 9 with pages of up to 64 tokens.  With
// larger ones it takes up to 10 too.)
#pragma once

#include <stdint.h>

// The kernel's loops have to stay small enough for the instruction cache, so
// what runs once per segment or less is a function of its own there (its
// arguments by value: by reference they would live in local memory).
#if defined(__CUDACC__)
#define DSPARK_HD __host__ __device__ __forceinline__
#define DSPARK_HD_CALL static __host__ __device__ __noinline__
#else
#define DSPARK_HD inline
#define DSPARK_HD_CALL static inline
#endif

namespace dspark {

constexpr int kKeyTile = 128;
constexpr int kRowTile = 64;

struct PlanInput {
    const int32_t* q_off;
    const int32_t* kv_len;
    int R, T, group, kv_heads;
    int64_t most;                  // max_pages * page
    int start;                     // length of an item besides its tiles
    uint32_t lengths;              // length of a tile, 5 bits each: up to 8, 16, 24, 32, 48, 64 rows (1 .. 31)
};
// Tokens that see the last `window` tokens, their own among them, and the first
// `sinks`.  unit: tokens that are left out together, a page's or a tile's, the
// smaller (a power of two); head: the sinks' tokens rounded up to units.
struct WindowPlan : PlanInput {
    int window, sinks, unit, head;
};
DSPARK_HD int plan_length(const PlanInput& p, int rows) {
    return (int)(p.lengths >> 5 * (rows <= 32 ? (rows - 1) / 8 : (rows <= 48 ? 4 : 5))) & 31;
}
// The longest tile that row tiles of up to `rows` rows have (lengths grow with them).
DSPARK_HD int plan_longest(const PlanInput& p, int64_t rows) { return plan_length(p, (int)(rows < kRowTile ? rows : kRowTile)); }

// A request's first row of the token axis, its new tokens and its keys, with
// values out of range clamped.
struct Request {
    int a, q_len, kv_len;
};
DSPARK_HD int plan_clamp(int64_t x, int64_t hi) { return (int)(x < 0 ? 0 : (x > hi ? hi : x)); }
DSPARK_HD Request plan_request(const PlanInput& p, int r) {
    const int a = plan_clamp(p.q_off[r], p.T), b = plan_clamp(p.q_off[r + 1], p.T);
    return Request{a, b > a ? b - a : 0, plan_clamp(p.kv_len[r], p.most < 0x7FFFFFFF ? p.most : 0x7FFFFFFF)};
}
DSPARK_HD int plan_row_tiles(const PlanInput& p, const Request& q) {
    return (int)(((int64_t)q.q_len * p.group + kRowTile - 1) / kRowTile);
}
// Keys that row rho (of q_len * group) sees.
DSPARK_HD_CALL int plan_row_keys(int group, int q_len, int kv_len, int64_t rho) {
    return plan_clamp((int64_t)kv_len - q_len + rho / group + 1, kv_len);
}
DSPARK_HD int plan_seen(const PlanInput& p, const Request& q, int64_t rho) {
    return plan_row_keys(p.group, q.q_len, q.kv_len, rho);
}
// Keys that row tile j reads (those of its last row), and how many key tiles they take.
DSPARK_HD int plan_tile_keys(const PlanInput& p, const Request& q, int j) {
    const int64_t rows = (int64_t)q.q_len * p.group, end = (int64_t)(j + 1) * kRowTile;
    // the last row tile's last row sees every key
    return end < rows ? plan_seen(p, q, end - 1) : q.kv_len;
}
// The new token that row tile j's first row belongs to.
DSPARK_HD int plan_first_token(const PlanInput& p, int j) { return j == 0 ? 0 : (int)((int64_t)j * kRowTile / p.group); }
// The first key that a window ending with new token i holds (may be negative).
DSPARK_HD int64_t plan_low(const WindowPlan& p, const Request& q, int i) {
    return (int64_t)q.kv_len - q.q_len + i - p.window + 1;
}
// The part below a tile of the tokens left out of a request's items: row tile 0
// leaves out what it can in units, the later ones whole tiles more, so that their
// number sums in closed form.
DSPARK_HD int plan_off(const WindowPlan& p, const Request& q) {
    const int64_t low = plan_low(p, q, 0);
    return low > p.head ? (int)(low - p.head) & (kKeyTile - 1) & ~(p.unit - 1) : 0;     // low <= kv_len
}
// Tokens between the sinks' pages and those of a row tile that begins with new token i.
DSPARK_HD int plan_gap(const PlanInput&, const Request&, int) { return 0; }
DSPARK_HD int plan_gap(const WindowPlan& p, const Request& q, int i) {
    const int off = plan_off(p, q);
    const int64_t n = plan_low(p, q, i) - p.head - off;
    return n > 0 ? ((int)n & ~(kKeyTile - 1)) + off : (n == 0 ? off : 0);
}
DSPARK_HD int plan_key_tiles(int keys) { return keys > 0 ? (keys - 1) / kKeyTile + 1 : 1; }
DSPARK_HD int plan_rows(const PlanInput& p, const Request& q, int j) {
    const int64_t rows = (int64_t)q.q_len * p.group - (int64_t)j * kRowTile;
    return (int)(rows < kRowTile ? rows : kRowTile);
}
// Where key tile t of an item begins, from the item's beginning (t = tiles:
// the item's length).
DSPARK_HD int64_t plan_place(const PlanInput& p, int length, int t) { return p.start + (int64_t)t * length; }
// The first key tile that begins at or after place x of an item.
DSPARK_HD int plan_tile_at(const PlanInput& p, int length, int64_t x, int tiles) {
    if (x <= p.start) return 0;
    if (x > plan_place(p, length, tiles - 1)) return tiles;
    return (int)(((uint32_t)(x - p.start) + (uint32_t)length - 1u) / (uint32_t)length);   // inside the item: below 2^30
}
// Length of a request's first n row tiles, all of them full and none its last:
// row tile j reads kv_len - q_len + floor((64 j + 63) / group) + 1 keys, so it
// takes max(0, floor((j + b) / 2 group)) + 1 key tiles, b = floor((63 +
// (kv_len - q_len) group) / 64), and the floors of a run from 0 sum in closed
// form.  (A walk over the row tiles, on every CTA before its first load, grew
// with a request's new tokens: 2048 of them, 32 heads to a group, over 4096 keys
// took 806 us and take 392; blocks of 1 to 17 tokens take the same.)
DSPARK_HD int64_t plan_floor_sum(int64_t y, uint32_t m) {                  // of floor(x / m), 0 <= x < y
    if (y <= 0) return 0;
    const uint32_t u = (uint32_t)y, d = u / m;                             // y <= 2 kv_len: 32 bits
    return (int64_t)d * (int32_t)(d - 1) / 2 * m + (int64_t)d * (u - d * m);
}
DSPARK_HD_CALL int64_t plan_before(int group, int start, int length, int q_len, int kv_len, int n) {
    const int64_t b = (63 + ((int64_t)kv_len - q_len) * group) >> 6;
    const uint32_t m = 2u * (uint32_t)group;
    return (int64_t)n * start + (n + plan_floor_sum(b + n, m) - plan_floor_sum(b, m)) * length;
}
DSPARK_HD int64_t plan_tiles_before(const PlanInput& p, const Request& q, int n) {
    return plan_before(p.group, p.start, plan_length(p, kRowTile), q.q_len, q.kv_len, n);
}
// Whole tiles that the first n row tiles leave out, each max(0, floor((j + b) / 2
// group)) of them: the same sum, b from the tokens left out before row tile 0.
DSPARK_HD_CALL int64_t plan_left_out_before(int group, int64_t ahead, int n) {
    const uint32_t m = 2u * (uint32_t)group;
    const int64_t b = ahead * group >> 6;
    return plan_floor_sum(b + n, m) - plan_floor_sum(b, m);
}
DSPARK_HD int64_t plan_tiles_before(const WindowPlan& p, const Request& q, int n) {
    const int off = plan_off(p, q);
    return plan_before(p.group, p.start, plan_length(p, kRowTile), q.q_len, q.kv_len - off, n) -
           plan_left_out_before(p.group, plan_low(p, q, 0) - p.head - off, n) * plan_length(p, kRowTile);
}
template <typename P>
DSPARK_HD_CALL int64_t plan_request_length(P p, int r) {
    const Request q = plan_request(p, r);
    const int n = plan_row_tiles(p, q);
    if (n == 0) return 0;
    const int64_t last = plan_place(p, plan_length(p, plan_rows(p, q, n - 1)), plan_key_tiles(q.kv_len - plan_gap(p, q, plan_first_token(p, n - 1))));
    return (plan_tiles_before(p, q, n - 1) + last) * p.kv_heads;
}
// The row tile that holds place x of request r's items: the last that begins at or before it.
template <typename P>
DSPARK_HD int plan_tile_of(const P& p, const Request& q, int64_t x) {
    int j = 0, upto = plan_row_tiles(p, q);
    while (upto - j > 1) {
        const int mid = j + (upto - j) / 2;
        if (plan_tiles_before(p, q, mid) * p.kv_heads <= x) j = mid;
        else upto = mid;
    }
    return j;
}
// How many of `grid` CTAs get a span: each span is at least as long as the
// widest gap between two tiles' beginnings, so that one begins in each (every
// CTA from an item's first to its last leaves a piece).
DSPARK_HD int plan_spans(const PlanInput& p, int64_t total, int grid) {
    const int64_t n = total / (p.start + plan_longest(p, (int64_t)p.T * p.group));
    return total == 0 ? 0 : (n < 1 ? 1 : (n < grid ? (int)n : grid));
}
// Where CTA c's span of n = plan_spans() begins (c = n: the end): floor(total c / n)
// without the product, which could pass 64 bits.
struct Span {
    int64_t begin, end;
};
DSPARK_HD_CALL Span plan_span(int64_t total, int c, int n) {
    const int64_t q = total / n;
    const uint32_t rest = (uint32_t)(total - q * n), u = (uint32_t)n;      // rest (c + 1) <= n^2: grids are far below 2^16
    return Span{q * c + rest * (uint32_t)c / u, q * (c + 1) + rest * ((uint32_t)c + 1u) / u};
}
DSPARK_HD int64_t plan_cut(int64_t total, int c, int n) { return c == n ? total : plan_span(total, c, n).begin; }
// The CTA whose span holds place g of the line: the largest c with total c / n < g + 1.
DSPARK_HD_CALL int plan_owner(int64_t total, int64_t g, int n) { return (int)(((g + 1) * n - 1) / total); }

// One CTA's piece of an item: key tiles [t0, t1) of tiles.
struct Segment {
    int r, j, h;
    int t0, t1, tiles;
    int keys;                      // keys the row tile reads
    int rows;                      // rows of the row tile
    int tok, head;                 // the first row's new token, and its place in the group
    int rest;                      // from the span's end to the beginning of the item's last tile (an unfinished item's: >= 0)
    Request q;
    int gap;                       // keys left out behind the sinks' (0 without a window)
};

// Row x of a row tile whose first row is (tok, head): its new token and its
// place in the group, in 32 bits.
DSPARK_HD void plan_row(int group, int tok, int head, int x, int& i, int& g) {
    const unsigned y = (unsigned)(head + x), d = y / (unsigned)group;
    i = tok + (int)d;
    g = (int)(y - d * (unsigned)group);
}
// Keys that new token i of a request sees.
DSPARK_HD int plan_token_keys(const Request& q, int i) {
    const int64_t n = (int64_t)q.kv_len - q.q_len + i + 1;
    return (int)(n < 0 ? 0 : n);                                  // i < q_len: at most kv_len
}

// Walks a span of the line.
struct Cursor {
    int r, j, h, t;
    int64_t end;                   // of the span, from the item's beginning
    Request q;

    // start inside request r, at place `skip` of its items, for a span of n
    template <typename P>
    DSPARK_HD void start(const P& p, int r_, int64_t skip, int64_t n) {
        r = r_;
        j = h = t = 0;
        end = 0;
        if (n <= 0) return;
        q = plan_request(p, r);
        j = plan_tile_of(p, q, skip);
        const int tiles = plan_key_tiles(plan_tile_keys(p, q, j) - plan_gap(p, q, plan_first_token(p, j))), length = plan_length(p, plan_rows(p, q, j));
        const int64_t item = plan_place(p, length, tiles);
        skip -= plan_tiles_before(p, q, j) * p.kv_heads;
        h = (int)(skip / item);
        skip -= h * item;
        t = plan_tile_at(p, length, skip, tiles);
        end = skip + n;
    }
    template <typename P>
    DSPARK_HD bool next(const P& p, Segment& s) {
        while (end > p.start) {                            // else no further tile begins in the span
            while (q.q_len == 0) q = plan_request(p, ++r); // the span goes on: a request with rows follows
            s.keys = plan_tile_keys(p, q, j);
            s.tok = plan_first_token(p, j);
            s.gap = plan_gap(p, q, s.tok);
            s.tiles = plan_key_tiles(s.keys - s.gap);
            s.rows = plan_rows(p, q, j);
            const int length = plan_length(p, s.rows);
            s.r = r;
            s.j = j;
            s.h = h;
            s.q = q;
            s.head = (int)((int64_t)j * kRowTile - (int64_t)s.tok * p.group);
            s.t0 = t;
            s.t1 = plan_tile_at(p, length, end, s.tiles);
            s.rest = (int)(plan_place(p, length, s.tiles - 1) - end);
            end -= plan_place(p, length, s.tiles);
            t = 0;
            if (end > 0 && ++h == p.kv_heads) {
                h = 0;
                if (++j == plan_row_tiles(p, q)) {
                    j = 0;
                    ++r;
                    q = Request{0, 0, 0};                  // read when the span reaches it
                    if (end > p.start) q = plan_request(p, r);
                }
            }
            if (s.t0 < s.t1) return true;
        }
        return false;
    }
};

}  // namespace dspark
