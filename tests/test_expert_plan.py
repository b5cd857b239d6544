"""Host arithmetic of the sort by expert and of the products with 4-bit weights (expert_plan.hpp, tile_choice.hpp): every
slot falls to one part, one workgroup's counters suffice, the workgroups hold every tile of every split of the rows, and a
launch's limit is told from one more."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HARNESS = r"""
#include <cstdio>
#include <vector>
#include "expert_plan.hpp"
#include "tile_choice.hpp"
using namespace tbg;
static int bad = 0;
#define CHECK(x, ...) do { if (!(x)) { std::printf("%s: ", #x); std::printf(__VA_ARGS__); std::printf("\n"); ++bad; } } while (0)
static uint64_t s = 88172645463325252ull;
static int64_t next(int64_t n) { s ^= s << 13; s ^= s >> 7; s ^= s << 17; return (int64_t)((s >> 11) % (uint64_t)n); }
static int64_t spread(int64_t hi) { return 1 + next(1 + next(hi)); }

static void plan(int64_t slots, int64_t groups) {
  const SortPlan p = plan_expert_sort(slots, groups);
  const long long a = slots, b = groups;
  CHECK(p.parts >= 1 && p.parts <= 256, "%lld %lld", a, b);
  CHECK(p.parts * p.part >= slots && (p.parts - 1) * p.part < slots + (slots == 0), "%lld %lld", a, b);
  CHECK(p.small ? p.parts == 1 && p.bytes == 0 : p.bytes >= p.parts * groups * 4 && p.part % 2048 == 0, "%lld %lld", a, b);
  // one workgroup: four slots a thread, as many waves as its 8192 counters serve
  int64_t waves = 16;
  while (waves > 1 && waves * groups > 8192) waves /= 2;
  CHECK(!p.small || slots <= waves * 256, "%lld %lld", a, b);
  CHECK(waves * groups <= 8192 && waves >= 2, "%lld %lld", a, b);
}

static void splits(int64_t groups, int64_t M, int64_t N) {
  std::vector<int64_t> sizes(groups, 0);
  for (int64_t left = M; left > 0;) {
    const int64_t n = 1 + next(left);
    sizes[next(groups)] += n;
    left -= n;
  }
  for (int kind = 0; kind < 2; ++kind) {
    const bool ragged = kind & 1;
    const TileChoice c = choose_w4(ragged ? groups : 0, M, N, 256);
    int64_t rows = 0;
    if (ragged) for (int64_t n : sizes) rows += tile_count(n, c.bm);
    else rows = tile_count(M, c.bm);
    CHECK(rows <= c.tiles_m, "groups %lld M %lld N %lld", (long long)groups, (long long)M, (long long)N);
    CHECK(c.tiles_n == tile_count(N, c.bn), "N %lld", (long long)N);
    CHECK(c.grid % 8 == 0 && c.grid >= c.tiles_m * c.tiles_n && c.fits(), "M %lld", (long long)M);
    CHECK(c.few ? c.bm == 16 && (c.bn == 16 || c.bn == 32 || c.bn == 64) : c.bn == 128 && (c.bm == 16 || c.bm == 32 || c.bm == 64),
          "%d x %d", c.bm, c.bn);
  }
}

int main() {
  for (int i = 0; i < 20000; ++i) plan(i % 3 ? spread(1 << 20) : spread(1 << 30), next(4097));
  for (int64_t n : {0, 1, 511, 512, 513, 4095, 4096, 4097, 1 << 30})
    for (int64_t e : {0, 1, 512, 513, 1024, 1025, 4095, 4096}) plan(n, e);
  for (int i = 0; i < 20000; ++i) splits(spread(200), spread(9000), spread(20000));
  // the most workgroups of one launch, and one tile more
  const int64_t most = (1 << 24) - 1, up = most / 8 * 8;
  CHECK(choose_w4(0, 64 * up, 128, 256).fits(), "dense");
  CHECK(!choose_w4(0, 64 * up + 1, 128, 256).fits(), "dense");
  CHECK(choose_w4(1, 64, 128 * up, 256).fits(), "ragged");
  CHECK(!choose_w4(1, 64, 128 * up + 1, 256).fits(), "ragged");
  std::printf("%s\n", bad ? "bad" : "ok");
  return bad != 0;
}
"""


def test_plans_and_choices(tmp_path):
    src = tmp_path / "plan.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "plan"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "tiled_bf16_gemm_amd", "csrc"),
                        str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout
