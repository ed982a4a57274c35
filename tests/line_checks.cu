// Host-side checks (built with nvcc as a host program, run by tests/test_line_arith.py) of the work line of
// the 4-bit store's split-K kernels, whose tiles have costs of their own:
//   * each tile is owned by one CTA, a unit's owners are consecutive, and each owns a tile of it, so that
//     its partial slots are counted exactly;
//   * the partial rows of a line's units fit the workspace laid out for both kernels;
//   * a workspace with a second shape holds each shape's own layout.
#include <algorithm>
#include <cstdio>
#include <vector>

#include "../varlen_gqa_attention_gb300/csrc/q4.cuh"

using namespace sdpa;

static int failures = 0;
#define CHECK(c)                                                \
  do {                                                          \
    if (!(c)) {                                                 \
      std::printf("FAIL %s:%d %s\n", __FILE__, __LINE__, #c);   \
      ++failures;                                               \
    }                                                           \
  } while (0)

static uint64_t state = 0x2545F4914F6CDD1Dull;
static uint64_t rnd(uint64_t n) {  // xorshift64*, below n
  state ^= state >> 12;
  state ^= state << 25;
  state ^= state >> 27;
  return (state * 0x2545F4914F6CDD1Dull >> 11) % n;
}

static void line(int kind, int most_rows) {
  const int nu = 1 + (int)rnd(60);
  std::vector<int64_t> base(nu), nt(nu), tw(nu);
  std::vector<int> rows(nu);
  const int64_t lead = lead_cost(kRouteSplitk, kind);
  int64_t Wp = 0;
  for (int u = 0; u < nu; ++u) {
    nt[u] = rnd(6) == 0 ? 0 : 1 + (int64_t)rnd(rnd(2) ? 4 : 400);
    rows[u] = 1 + (int)rnd(rnd(2) ? 8 : most_rows);
    tw[u] = tile_cost(kRouteSplitk, rows[u], kind);
    base[u] = Wp;
    Wp += nt[u] > 0 ? lead + nt[u] * tw[u] : 0;
  }
  if (Wp == 0) return;
  const int64_t G = 1 + (int64_t)rnd(500), Gp = phase_ctas(G, Wp, kRouteSplitk, kind);
  CHECK(Gp >= 1 && Gp <= G);
  int64_t partial = 0;
  for (int u = 0; u < nu; ++u) {
    if (nt[u] == 0) continue;
    const int64_t k0 = base[u] + lead;
    std::vector<int64_t> owner(nt[u], -1);
    for (int64_t g = 0; g < Gp; ++g) {
      int64_t ta, tb;
      line_tiles(sk_start(g, Wp, Gp), sk_start(g + 1, Wp, Gp), k0, nt[u], tw[u], &ta, &tb);
      for (int64_t t = ta; t < tb; ++t) {
        CHECK(owner[t] == -1);
        owner[t] = g;
      }
    }
    const int64_t g0 = sk_owner(k0, Wp, Gp), g1 = sk_owner(k0 + (nt[u] - 1) * tw[u], Wp, Gp);
    CHECK(owner[0] == g0 && owner[nt[u] - 1] == g1);
    for (int64_t t = 0; t < nt[u]; ++t) {
      CHECK(owner[t] >= 0);
      if (t > 0) CHECK(owner[t] == owner[t - 1] || owner[t] == owner[t - 1] + 1);
    }
    if (g1 > g0) partial += (g1 - g0 + 1) * rows[u];
  }
  CHECK(partial <= part_cap(nu, G, most_rows));
}

int main() {
  for (int i = 0; i < 4000; ++i) {
    line(kSkQ4Few, kSplitkRows);
    line(kSkQ4Tile, kQ4TileRows);
  }
  // the costliest tile of a kind is what phase_ctas shares out at least
  for (int rows = 1; rows <= kSplitkRows; ++rows) CHECK(tile_cost(kRouteSplitk, rows, kSkQ4Few) <= 16);
  for (int rows = 1; rows <= kQ4TileRows; ++rows) CHECK(tile_cost(kRouteSplitk, rows, kSkQ4Tile) <= 5);
  CHECK(phase_ctas(1000, 16 * 7 + 15, kRouteSplitk, kSkQ4Few) == 7);
  CHECK(phase_ctas(1000, 5 * 7 + 4, kRouteSplitk, kSkQ4Tile) == 7);

  for (int i = 0; i < 4000; ++i) {
    const int Hkv = 1 << (int)rnd(5), Hq = Hkv * (1 + (int)rnd(32)), S = (int)rnd(100), D = rnd(2) ? 64 : 128;
    const int64_t T = (int64_t)rnd(rnd(2) ? 200 : 20000);
    const SkShape tile{kQ4TileRows, kQ4TileKeys, kSkQ4Tile, 152};
    Workspace w{};
    char* at = reinterpret_cast<char*>(uintptr_t{1} << 40);
    const size_t n = layout_workspace(at, T, Hq, Hkv, D, S, 304, 152, &w, true, &tile);
    CHECK(n >= layout_workspace(nullptr, T, Hq, Hkv, D, S, 304, 152, nullptr));
    CHECK(w.unit_cap[1] >= unit_cap(T, Hq, Hkv, S, kSplitkRows) && w.unit_cap[1] >= unit_cap(T, Hq, Hkv, S, kQ4TileRows));
    CHECK(w.part_cap[1] >= part_cap(unit_cap(T, Hq, Hkv, S, kSplitkRows), 304, kSplitkRows));
    CHECK(w.part_cap[1] >= part_cap(unit_cap(T, Hq, Hkv, S, kQ4TileRows), 152, kQ4TileRows));
    CHECK((char*)w.unit_done + 4 * w.unit_cap[1] <= at + n);
    CHECK((char*)w.part_ml[1] - (char*)w.first_unit[1] >= 4 * kMaxPhases * 304);
    CHECK((char*)w.part_o[1] - (char*)w.part_ml[1] >= (int64_t)(8 * w.part_cap[1]));
    CHECK((char*)w.units[2] - (char*)w.part_o[1] >= (int64_t)(4 * D * w.part_cap[1]));
  }
  std::printf("failures %d\n", failures);
  return failures != 0;
}
