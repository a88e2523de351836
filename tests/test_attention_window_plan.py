"""The work split of paged attention with a window (csrc/attn_plan.h), compiled
for the host: over random batches, values out of range among them, the segments
cover the keys that some row of the item sees and little else, page by page and
counted row by row, once each, and every index stays in range."""
import shutil
import subprocess

import pytest

from speculative_decoding_drafting_gb300 import _build

PROGRAM = r"""
#include <cstdio>
#include <map>
#include <random>
#include <tuple>
#include <vector>
#include "attn_plan.h"
using namespace dspark;

#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s (trial %d)\n", __LINE__, #c, trial); return 1; } } while (0)

int main() {
    std::mt19937_64 rng(11);
    auto pick = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
    for (int trial = 0; trial < 4000; ++trial) {
        const int R = (int)pick(1, trial % 5 == 0 ? 200 : 9), group = (int)pick(1, trial % 3 == 0 ? 128 : 8);
        const int kv_heads = (int)pick(1, 9), page = 16 << pick(0, 4), max_pages = (int)pick(1, 400);
        const int64_t most = (int64_t)page * max_pages;
        std::vector<int32_t> off(R + 1), len(R);
        const bool wild = trial % 4 == 3;
        int at = wild ? (int)pick(-5, 5) : 0;
        for (int r = 0; r <= R; ++r) {
            off[r] = at;
            at += (int)pick(wild ? -3 : 0, trial % 7 == 0 ? 400 : 6);
        }
        const int T = wild ? (int)pick(0, 40) : off[R];
        for (int r = 0; r < R; ++r) {
            len[r] = (int)pick(0, trial % 2 ? most : (most < 300 ? most : 300));
            if (wild && pick(0, 3) == 0) len[r] = pick(0, 1) ? (int)pick(-2147483647 - 1ll, -1) : (int)pick(most, 2147483647);
        }
        int start = (int)pick(0, 9), length = (int)pick(1, 5);
        uint32_t lengths = 0;
        for (int k = 0; k < 6; ++k) {
            lengths |= (uint32_t)length << (5 * k);
            length += (int)pick(0, 5);
        }
        WindowPlan p;
        static_cast<PlanInput&>(p) = PlanInput{off.data(), len.data(), R, T, group, kv_heads, most, start, lengths};
        p.window = (int)pick(1, trial % 8 == 0 ? 1 << 30 : (trial % 2 ? 5000 : 200));
        p.sinks = trial % 3 ? (int)pick(0, trial % 9 ? 20 : 700) : 0;
        p.unit = page < kKeyTile ? page : kKeyTile;
        p.head = (p.sinks + p.unit - 1) / p.unit * p.unit;
        int64_t total = 0;
        std::vector<int64_t> first(R);
        for (int r = 0; r < R; ++r) {
            first[r] = total;
            total += plan_request_length(p, r);
        }
        const int n = plan_spans(p, total, (int)pick(1, 152));
        if (total == 0) { CHECK(n == 0); continue; }
        std::map<std::tuple<int, int, int>, int> done, last;
        std::map<std::tuple<int, int, int>, std::pair<int, int>> shape;
        for (int c = 0; c < n; ++c) {
            const int64_t b = plan_cut(total, c, n), e = plan_cut(total, c + 1, n);
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
                CHECK(s.rows >= 1 && s.rows <= kRowTile && (int64_t)s.j * kRowTile + s.rows <= (int64_t)s.q.q_len * group);
                CHECK(s.keys >= 0 && s.keys <= s.q.kv_len && s.keys <= most);
                CHECK(0 <= s.t0 && s.t0 < s.t1 && s.t1 <= s.tiles && s.gap >= 0 && s.gap % p.unit == 0);
                // the item's units are those that hold a key of a row, and the sinks'
                auto physical = [&](int v) { return v >= p.head ? v + s.gap : v; };
                std::vector<char> need((s.keys + p.unit - 1) / p.unit + 1, 0);
                int64_t low = 1ll << 40;
                for (int x = 0; x < s.rows; ++x) {
                    int i, g;
                    plan_row(group, s.tok, s.head, x, i, g);
                    const int64_t pos = (int64_t)s.q.kv_len - s.q.q_len + i, from = pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
                    if (pos >= 0 && from < low) low = from;
                    for (int64_t k = from / p.unit * p.unit; k <= pos; k += p.unit) need[k / p.unit] = 1;
                    for (int64_t k = 0; k < p.sinks && k <= pos; k += p.unit) need[k / p.unit] = 1;
                }
                int covered = 0, extra = 0;
                for (int v = 0; v < s.tiles * kKeyTile; v += p.unit) {
                    const int k = physical(v);
                    if (k >= s.keys) { CHECK(v / kKeyTile == s.tiles - 1); continue; }
                    covered += need[k / p.unit];
                    extra += !need[k / p.unit];
                }
                int needed = 0;
                for (char x : need) needed += x;
                CHECK(covered == needed);
                // row tile 0 takes nothing else, the later ones less than a tile
                CHECK(extra * p.unit < (s.j == 0 ? p.unit : kKeyTile));
                const auto id = std::make_tuple(s.r, s.j, s.h);
                CHECK(done[id] == s.t0);
                CHECK(s.t0 == 0 || shape[id] == std::make_pair(s.tiles, s.gap));
                shape[id] = std::make_pair(s.tiles, s.gap);
                done[id] = s.t1;
                ++pieces;
                CHECK(s.t0 == 0 || pieces == 1);
                if (s.t0 == 0 && s.t1 < s.tiles) {
                    CHECK(s.rest >= 0);
                    const int owner = plan_owner(total, e + s.rest, n);
                    CHECK(owner > c && owner < n);
                    last[id] = owner;
                }
                if (s.t0 > 0) {
                    CHECK(c <= last[id]);
                    CHECK((s.t1 == s.tiles) == (c == last[id]));
                }
                tail = s.t1 < s.tiles;
            }
            CHECK(pieces > 0);
        }
        for (int r = 0; r < R; ++r) {
            const Request q = plan_request(p, r);
            for (int j = 0; j < plan_row_tiles(p, q); ++j)
                for (int h = 0; h < kv_heads; ++h) {
                    const auto id = std::make_tuple(r, j, h);
                    CHECK(done[id] > 0 && done[id] == shape[id].first);
                }
        }
    }
    // long requests: the closed form against the sum over the row tiles
    for (int trial = 0; trial < 400; ++trial) {
        const int group = (int)pick(1, 128), q_len = (int)pick(1, 3000), kv = (int)pick(0, 1 << 30);
        int32_t off[2] = {0, q_len}, len[1] = {kv};
        WindowPlan p;
        static_cast<PlanInput&>(p) = PlanInput{off, len, 1, q_len, group, 1, 1 << 30, 3, 0x02108421u};
        p.window = (int)pick(1, trial % 2 ? 1 << 30 : 5000);
        p.sinks = (int)pick(0, 1000);
        p.unit = 16 << pick(0, 3);
        p.head = (p.sinks + p.unit - 1) / p.unit * p.unit;
        const Request q = plan_request(p, 0);
        int64_t sum = 0;
        const int n = plan_row_tiles(p, q);
        for (int j = 0; j < n; ++j) {
            CHECK(sum == plan_tiles_before(p, q, j));
            const int tiles = plan_key_tiles(plan_tile_keys(p, q, j) - plan_gap(p, q, plan_first_token(p, j)));
            CHECK(tiles >= 1);
            sum += plan_place(p, plan_length(p, plan_rows(p, q, j)), tiles);
        }
        CHECK(sum == plan_request_length(p, 0));
    }
    std::printf("ok\n");
    return 0;
}
"""


def test_segments_cover_what_the_windows_need(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-O1", "-g", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", _build.CSRC,
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
