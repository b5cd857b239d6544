"""The choice of kernels and workgroups of the ragged and the 4-bit products
(tiled_bf16_gemm_amd/csrc/tile_choice.hpp), on the host: the workgroups hold every tile of every split of
the rows, and the most that one launch takes (2^24 - 1) is told from one more, for every kernel."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HARNESS = r"""
#include <cstdio>
#include <vector>
#include "tile_choice.hpp"
using namespace tbg;
static int bad = 0;
#define CHECK(x, ...) do { if (!(x)) { std::printf("%s: ", #x); std::printf(__VA_ARGS__); std::printf("\n"); ++bad; } } while (0)
static uint64_t s = 88172645463325252ull;
static int64_t next(int64_t n) { s ^= s << 13; s ^= s >> 7; s ^= s << 17; return (int64_t)((s >> 11) % (uint64_t)n); }
static int64_t spread(int64_t hi) { return 1 + next(1 + next(hi)); }

// Workgroups against the tiles of a random split.
static void splits(int64_t groups, int64_t M, int64_t N, int64_t K) {
  std::vector<int64_t> sizes(groups, 0);
  for (int64_t left = M, g; left > 0;) {
    g = next(groups);
    const int64_t n = 1 + next(left);
    sizes[g] += n;
    left -= n;
  }
  for (int kind = 0; kind < 3; ++kind) {
    const TileChoice c = kind < 2 ? choose_grouped(groups, M, N, K, kind == 0, 256) : choose_mx4(groups, M, N, K, 256);
    int64_t rows = 0;
    for (int64_t n : sizes) rows += tile_count(n, c.bm);
    CHECK(rows <= c.tiles_m, "kind %d groups %lld M %lld", kind, (long long)groups, (long long)M);
    CHECK(c.tiles_n == tile_count(N, c.bn), "kind %d N %lld", kind, (long long)N);
    CHECK(c.fits(), "kind %d M %lld N %lld", kind, (long long)M, (long long)N);
    CHECK(c.grid % 8 == 0 && (c.walks || c.grid >= c.tiles_m * c.tiles_n), "kind %d grid %lld", kind, (long long)c.grid);
    CHECK(!c.few || (M <= 16 * (groups < M ? groups : M) && kind != 1), "kind %d M %lld", kind, (long long)M);
    CHECK((c.bm == 256) == c.walks || kind < 2, "kind %d", kind);
  }
}

// Every tile of every group falls to one workgroup (the numbering of grad_tile in ragged.hpp).
static void grads(int64_t groups, int64_t M, int64_t P, int64_t Q) {
  const TileChoice c = choose_wgrad(groups, M, P, Q, 256);
  CHECK(c.fits(), "P %lld Q %lld", (long long)P, (long long)Q);
  std::vector<char> seen(groups * c.tiles_m * c.tiles_n, 0);
  int64_t found = 0;
  for (int64_t bid = 0; bid < c.grid; ++bid) {
    const int64_t x = bid & 7, i = bid >> 3, id = i / c.per_xcd * (8 * c.per_xcd) + x * c.per_xcd + i % c.per_xcd;
    if (id < (int64_t)seen.size() && !seen[id]) seen[id] = 1, ++found;
  }
  CHECK(found == (int64_t)seen.size(), "groups %lld P %lld Q %lld: %lld tiles", (long long)groups, (long long)P, (long long)Q,
        (long long)found);
}

int main() {
  for (int i = 0; i < 20000; ++i) splits(spread(200), spread(9000), spread(9000), 32 * spread(300));
  for (int i = 0; i < 2000; ++i) grads(spread(200), spread(20000), spread(4000), spread(4000));
  const int64_t most = (1 << 24) - 1, up = 1ll << 30;
  // 64 columns a workgroup, ragged: the last whole eighth, then one tile more
  for (int nk = 0; nk < 2; ++nk) {
    TileChoice c = choose_grouped(1, 1, 64 * (most - 7), 8, nk, 256);
    CHECK(!c.few && c.bm == 64 && c.grid == most - 7 && c.fits(), "grid %lld", (long long)c.grid);
    c = choose_grouped(1, 1, 64 * (most - 7) + 1, 8, nk, 256);
    CHECK(c.grid == most + 1 && !c.fits(), "grid %lld", (long long)c.grid);
    c = choose_grouped(1, 1, up, 8, nk, 256);
    CHECK(!c.fits(), "grid %lld", (long long)c.grid);
    c = choose_grouped(4096, up, up, 8, nk, 256);
    CHECK(!c.fits() && c.grid > most, "grid %lld", (long long)c.grid);
  }
  // 32 and 64 rows in 4 bits, dense: exactly the most, then one more
  for (int64_t M : {1, 32, 33, 64}) {
    TileChoice c = choose_mx4(0, M, 64 * most, 32, 256);
    CHECK(!c.few && c.bn == 64 && c.grid == most && c.fits(), "M %lld grid %lld", (long long)M, (long long)c.grid);
    c = choose_mx4(0, M, 64 * most + 1, 32, 256);
    CHECK(c.grid == most + 1 && !c.fits(), "M %lld grid %lld", (long long)M, (long long)c.grid);
    c = choose_mx4(1, M, 64 * (most - 7) + 1, 32, 256);
    CHECK(c.grid == most + 1 && !c.fits(), "M %lld grid %lld", (long long)M, (long long)c.grid);
  }
  // stages of the 64-column tiles: up to 1.5 workgroups a compute unit, and from K = 8192 on
  for (int64_t M : {20, 60}) {
    CHECK(choose_mx4(0, M, 64 * 384, 4096, 256).stages == 4 && choose_mx4(0, M, 64 * 385, 4096, 256).stages == 2, "M %d", (int)M);
    CHECK(choose_mx4(0, M, 64 * 4000, 8160, 256).stages == 2 && choose_mx4(0, M, 64 * 4000, 8192, 256).stages == 4, "M %d", (int)M);
    CHECK(choose_mx4(16, 16 * M, 64 * 24, 4096, 256).stages == 4 && choose_mx4(16, 16 * M, 64 * 25, 4096, 256).stages == 2, "M %d", (int)M);
  }
  // the walking tile: any number of tiles that 32 bits hold, on as many workgroups as compute units
  for (int64_t groups : {0, 3}) {
    TileChoice c = choose_mx4(groups, 1 << 22, 1 << 22, 8192, 256);
    CHECK(c.walks && c.grid == 256 && c.fits(), "grid %lld", (long long)c.grid);
    c = choose_mx4(groups, up, up, 8192, 256);
    CHECK(c.walks && !c.fits(), "tiles %lld x %lld", (long long)c.tiles_m, (long long)c.tiles_n);
  }
  // the weight gradient: 2^24 - 4096 and 2^24 tiles of 256 x 256
  TileChoice c = choose_wgrad(4095, 1 << 24, 256 * 64, 256 * 64, 256);
  CHECK(c.bm == 256 && c.grid == 4095 * 4096 && c.fits(), "tile %d grid %lld", c.bm, (long long)c.grid);
  c = choose_wgrad(4096, 1 << 24, 256 * 64, 256 * 64, 256);
  CHECK(c.bm == 256 && c.grid == most + 1 && !c.fits(), "tile %d grid %lld", c.bm, (long long)c.grid);
  c = choose_wgrad(4096, up, up, up, 256);
  CHECK(!c.fits(), "grid %lld", (long long)c.grid);
  // groups in the order of their rows: 2 to 64 of 1024 rows on average
  CHECK(choose_wgrad(64, 65536, 99, 99, 256).by_rows && choose_wgrad(2, 2048, 99, 99, 256).by_rows, "by rows");
  CHECK(!choose_wgrad(64, 65535, 99, 99, 256).by_rows && !choose_wgrad(65, 1 << 20, 99, 99, 256).by_rows, "by number");
  CHECK(!choose_wgrad(1, 1 << 20, 99, 99, 256).by_rows, "one group");
  // both repacks of a call: 2^24 - 1 workgroups of 256 chunks together, and one chunk more
  const uint64_t all = (uint64_t)most * 256;
  CHECK(one_pack_launch(all, 0) && one_pack_launch(0, all) && one_pack_launch(all - 512, 257), "the most");
  CHECK(!one_pack_launch(all + 1, 0) && !one_pack_launch(all, 1) && !one_pack_launch(all - 512, 513), "one more");
  CHECK(!one_pack_launch(all / 2 + 256, all / 2 + 256) && !one_pack_launch(~0ull / 4, ~0ull / 4), "far more");
  std::printf("%d problems\n", bad);
  return bad != 0;
}
"""


def test_workgroups_hold_every_tile_and_the_most_are_told_from_one_more(tmp_path):
    src = tmp_path / "tile_choice_check.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "tile_choice_check"
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "tiled_bf16_gemm_amd", "csrc"),
                        str(src), "-o", str(exe)], capture_output=True, text=True)
    if r.returncode != 0:
        pytest.fail(r.stderr)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "0 problems", r.stdout[-3000:]
