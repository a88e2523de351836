"""The work split of paged attention (csrc/attn_plan.h), compiled for the
host: over random batches, values out of range among them, the CTAs' segments
cover every item's key tiles exactly once and every index stays in range."""
import os
import shutil
import subprocess

import pytest

from speculative_decoding_drafting_gb300 import _build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <tuple>
#include <vector>
#include "attn_plan.h"
using namespace dspark;

#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s (trial %d)\n", __LINE__, #c, trial); return 1; } } while (0)

int main() {
    std::mt19937_64 rng(7);
    auto pick = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
    for (int trial = 0; trial < 4000; ++trial) {
        const int R = (int)pick(1, trial % 5 == 0 ? 300 : 9), group = (int)pick(1, trial % 3 == 0 ? 128 : 8);
        const int kv_heads = (int)pick(1, 9), page = 16 << pick(0, 4), max_pages = (int)pick(1, 400);
        const int64_t most = (int64_t)page * max_pages;
        std::vector<int32_t> off(R + 1), len(R);
        const bool wild = trial % 4 == 3;
        int at = wild ? (int)pick(-5, 5) : 0;
        for (int r = 0; r <= R; ++r) {
            off[r] = at;
            at += (int)pick(wild ? -3 : 0, trial % 7 == 0 ? 90 : 6);
        }
        const int T = wild ? (int)pick(0, 40) : off[R];
        for (int r = 0; r < R; ++r) {
            len[r] = (int)pick(0, trial % 2 ? most : (most < 300 ? most : 300));
            if (wild && pick(0, 3) == 0) len[r] = pick(0, 1) ? (int)pick(-2147483647 - 1ll, -1) : (int)pick(most, 2147483647);
        }
        // any lengths that grow with the rows
        int start = (int)pick(0, 9), length = (int)pick(1, 5);
        uint32_t lengths = 0;
        for (int k = 0; k < 6; ++k) {
            lengths |= (uint32_t)length << (5 * k);
            length += (int)pick(0, 5);
        }
        if (trial % 6 == 5) {                               // every tile as long as another, as the simplest case
            start = 0;
            lengths = 0x02108421u;
        }
        const PlanInput p{off.data(), len.data(), R, T, group, kv_heads, most, start, lengths};
        int64_t total = 0;
        std::vector<int64_t> first(R);
        for (int r = 0; r < R; ++r) {
            first[r] = total;
            total += plan_request_length(p, r);
        }
        const int n = plan_spans(p, total, (int)pick(1, 152));
        if (total == 0) { CHECK(n == 0); continue; }
        CHECK(plan_cut(total, 0, n) == 0 && plan_cut(total, n, n) == total);
        std::map<std::tuple<int, int, int>, int> done, last;
        int64_t seen_tiles = 0;
        for (int c = 0; c < n; ++c) {
            const int64_t b = plan_cut(total, c, n), e = plan_cut(total, c + 1, n);
            CHECK(b < e && e - b <= total / n + 1);
            int r = 0;
            while (!(first[r] <= b && b < first[r] + plan_request_length(p, r))) CHECK(++r < R);
            Cursor cur;
            cur.start(p, r, b - first[r], e - b);
            Segment s;
            bool tail = false;
            int pieces = 0;
            while (cur.next(p, s)) {
                CHECK(!tail);
                CHECK(s.r >= 0 && s.r < R && s.h >= 0 && s.h < kv_heads);
                CHECK(s.q.a >= 0 && s.q.q_len > 0 && s.q.a + s.q.q_len <= T);
                CHECK(s.rows >= 1 && s.rows <= kRowTile);
                CHECK((int64_t)s.j * kRowTile + s.rows <= (int64_t)s.q.q_len * group);
                CHECK(s.keys >= 0 && s.keys <= s.q.kv_len && s.keys <= most);
                CHECK(0 <= s.t0 && s.t0 < s.t1 && s.t1 <= s.tiles);
                CHECK(s.keys <= (int64_t)s.tiles * kKeyTile && (s.tiles == 1 || (s.tiles - 1) * (int64_t)kKeyTile < s.keys));
                for (int x = 0; x < s.rows; ++x) {
                    const int seen = plan_seen(p, s.q, (int64_t)s.j * kRowTile + x);
                    CHECK(seen >= 0 && seen <= s.keys);
                    int i, g;
                    plan_row(group, s.tok, s.head, x, i, g);
                    CHECK((int64_t)i * group + g == (int64_t)s.j * kRowTile + x && g < group && i < s.q.q_len);
                    CHECK(plan_token_keys(s.q, i) == seen);
                }
                int& d = done[std::make_tuple(s.r, s.j, s.h)];
                CHECK(d == s.t0);
                d = s.t1;
                ++pieces;
                CHECK(s.t0 == 0 || pieces == 1);            // only a span's first piece begins inside its item
                if (s.t0 == 0 && s.t1 < s.tiles) {          // the piece that describes the join
                    CHECK(s.rest >= 0);
                    const int owner = plan_owner(total, e + s.rest, n);
                    CHECK(owner > c && owner < n);
                    CHECK(plan_cut(total, owner, n) <= e + s.rest && e + s.rest < plan_cut(total, owner + 1, n));
                    last[std::make_tuple(s.r, s.j, s.h)] = owner;
                }
                if (s.t0 > 0) {                             // every CTA from the first to the last has a piece
                    CHECK(c <= last[std::make_tuple(s.r, s.j, s.h)]);
                    CHECK((s.t1 == s.tiles) == (c == last[std::make_tuple(s.r, s.j, s.h)]));
                }
                tail = s.t1 < s.tiles;
            }
            CHECK(pieces > 0);
            seen_tiles += e - b;
        }
        CHECK(seen_tiles == total);
        for (int r = 0; r < R; ++r) {
            const Request q = plan_request(p, r);
            for (int j = 0; j < plan_row_tiles(p, q); ++j)
                for (int h = 0; h < kv_heads; ++h)
                    CHECK(done[std::make_tuple(r, j, h)] == plan_key_tiles(plan_tile_keys(p, q, j)));
        }
    }
    std::printf("ok\n");
    return 0;
}
"""


def test_segments_cover_every_item_once(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-O1", "-g", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", _build.CSRC,
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
