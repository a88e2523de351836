"""Requests of many new tokens in the work split of paged attention
(csrc/attn_plan.h, compiled for the host): the closed form of their length and
of where a span begins agrees with a walk over the row tiles, and takes no time
that grows with them."""
import shutil
import subprocess

import pytest

from speculative_decoding_drafting_gb300 import _build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include "attn_plan.h"
using namespace dspark;

#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s (trial %d)\n", __LINE__, #c, trial); return 1; } } while (0)

int main() {
    std::mt19937_64 rng(11);
    auto pick = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
    for (int trial = 0; trial < 3000; ++trial) {
        const int group = (int)pick(1, trial % 3 ? 128 : 9), kv_heads = (int)pick(1, 5);
        const int q_len = (int)pick(1, trial % 4 ? 300 : 6000);
        int32_t len = (int32_t)(trial % 2 ? pick(0, 9000) : pick(q_len, q_len + 5000));
        const int32_t off[2] = {0, q_len};
        uint32_t lengths = 0;
        int length = (int)pick(1, 5);
        for (int k = 0; k < 6; ++k) {
            lengths |= (uint32_t)length << (5 * k);
            length += (int)pick(0, 5);
        }
        const PlanInput p{off, &len, 1, q_len, group, kv_heads, int64_t(1) << 40, (int)pick(0, 12), lengths};
        const Request q = plan_request(p, 0);
        const int n = plan_row_tiles(p, q);
        int64_t sum = 0;
        const int64_t total = plan_request_length(p, 0);
        for (int j = 0; j < n; ++j) {
            const int tiles = plan_key_tiles(plan_tile_keys(p, q, j));
            const int64_t item = plan_place(p, plan_length(p, plan_rows(p, q, j)), tiles);
            if (n < 20 || j % (n / 9) == 0 || j == n - 1) {
                const int h = (int)pick(0, kv_heads - 1);
                const int64_t x = pick(0, item - 1);
                Cursor c;
                c.start(p, 0, sum * kv_heads + h * item + x, 1);
                CHECK(c.j == j && c.h == h && c.end == x + 1);
                CHECK(c.t == plan_tile_at(p, plan_length(p, plan_rows(p, q, j)), x, tiles));
            }
            sum += item;
        }
        CHECK(total == sum * kv_heads);
    }
    // 2^25 row tiles of one request
    const int trial = -1;
    const int32_t off[2] = {0, 1 << 24}, len = (1 << 24) + 77777;
    const PlanInput p{off, &len, 1, 1 << 24, 128, 4, int64_t(1) << 40, 8, 0x0E629084u};
    int64_t sum = 0;
    for (int i = 0; i < 2000; ++i) {
        sum ^= plan_request_length(p, 0);
        Cursor c;
        c.start(p, 0, plan_request_length(p, 0) - 1 - i, 1);
        CHECK(c.j == (1 << 25) - 1 || c.j > 0);
    }
    std::printf("ok %lld\n", (long long)sum);
    return 0;
}
"""


def test_long_requests_take_no_walk(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-O1", "-g", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", _build.CSRC,
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
