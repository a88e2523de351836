// attn_plan.h -- how paged attention splits its work (plain C++, also
// compiled for the host, where its index ranges are checked).
//
// An item is one row tile of one request and one key-value head: up to
// kRowTile of the request's rows (row = new token x query heads of the group,
// heads fastest) over the keys that its last row sees, in tiles of kKeyTile
// keys, at least one.  Items are numbered request, row tile, head; the tiles
// of all items form one line, which is cut into equal spans, one per CTA, so
// that requests of any mix of lengths load the device evenly.  An item that a
// cut goes through leaves one partial result per piece.
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
};

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
DSPARK_HD int plan_seen(const PlanInput& p, const Request& q, int64_t rho) {
    return plan_clamp((int64_t)q.kv_len - q.q_len + rho / p.group + 1, q.kv_len);
}
// Keys that row tile j reads, and how many key tiles they take.
DSPARK_HD_CALL int plan_inner_keys(int group, int q_len, int kv_len, int j) {
    const int64_t n = (int64_t)kv_len - q_len + (((int64_t)(j + 1) * kRowTile - 1) / group) + 1;
    return plan_clamp(n, kv_len);
}
DSPARK_HD int plan_tile_keys(const PlanInput& p, const Request& q, int j) {
    const int64_t rows = (int64_t)q.q_len * p.group, end = (int64_t)(j + 1) * kRowTile;
    // the last row tile's last row sees every key
    return end < rows ? plan_inner_keys(p.group, q.q_len, q.kv_len, j) : q.kv_len;
}
DSPARK_HD int plan_key_tiles(int keys) { return keys > 0 ? (keys - 1) / kKeyTile + 1 : 1; }
DSPARK_HD_CALL int64_t plan_request_tiles(PlanInput p, int r) {
    const Request q = plan_request(p, r);
    const int n = plan_row_tiles(p, q);
    int64_t sum = 0;
    for (int j = 0; j < n; ++j) sum += plan_key_tiles(plan_tile_keys(p, q, j));
    return sum * p.kv_heads;
}
// How many of `grid` CTAs get a span: none is left empty between two others,
// since every CTA from an item's first to its last leaves a piece.
DSPARK_HD int plan_spans(int64_t total, int grid) { return total < grid ? (int)total : grid; }
// First tile of CTA c of n = plan_spans() (c = n: the end): floor(total c / n)
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
// The CTA whose span holds tile g: the largest c with total c / n < g + 1.
DSPARK_HD_CALL int plan_owner(int64_t total, int64_t g, int n) { return (int)(((g + 1) * n - 1) / total); }

// One CTA's piece of an item: key tiles [t0, t1) of tiles.
struct Segment {
    int r, j, h;
    int t0, t1, tiles;
    int keys;                      // keys the row tile reads
    int rows;                      // rows of the row tile
    int tok, head;                 // the first row's new token, and its place in the group
    Request q;
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

// Walks a span of the line of tiles.
struct Cursor {
    int r, j, h, t;
    int64_t left;
    Request q;

    // start inside request r, `skip` tiles after its first
    DSPARK_HD void start(const PlanInput& p, int r_, int64_t skip, int64_t n) {
        r = r_;
        j = h = t = 0;
        left = n;
        if (n <= 0) return;
        q = plan_request(p, r);
        for (;; ++j) {
            const int tiles = plan_key_tiles(plan_tile_keys(p, q, j));
            if (skip < (int64_t)tiles * p.kv_heads) {
                h = (int)(skip / tiles);
                t = (int)(skip % tiles);
                return;
            }
            skip -= (int64_t)tiles * p.kv_heads;
        }
    }
    DSPARK_HD bool next(const PlanInput& p, Segment& s) {
        if (left <= 0) return false;
        while (q.q_len == 0) q = plan_request(p, ++r);     // left > 0: a request with rows follows
        const int64_t rows = (int64_t)q.q_len * p.group - (int64_t)j * kRowTile;
        s.r = r;
        s.j = j;
        s.h = h;
        s.q = q;
        s.keys = plan_tile_keys(p, q, j);
        s.tiles = plan_key_tiles(s.keys);
        s.rows = (int)(rows < kRowTile ? rows : kRowTile);
        s.tok = (int)((int64_t)j * kRowTile / p.group);
        s.head = (int)((int64_t)j * kRowTile - (int64_t)s.tok * p.group);
        s.t0 = t;
        s.t1 = (int)(s.tiles - t < left ? s.tiles : t + left);
        left -= s.t1 - s.t0;
        t = 0;
        if (left > 0 && ++h == p.kv_heads) {
            h = 0;
            if (++j == plan_row_tiles(p, q)) {
                j = 0;
                ++r;
                q = plan_request(p, r);
            }
        }
        return true;
    }
};

}  // namespace dspark
