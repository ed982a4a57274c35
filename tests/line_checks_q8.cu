// Host-side checks (built with nvcc as a host program, run by tests/test_line_arith_q8.py) of the work line of the
// 8-bit store's split-K kernel for few rows, and of the small scheduler's bound for units of 128 rows:
//   * each tile is owned by one CTA, a unit's owners are consecutive, and each owns a tile of it, so that
//     its partial slots are counted exactly;
//   * the partial rows of a line's units fit the workspace;
//   * a call that the small scheduler admits has no more units than threads.
#include <algorithm>
#include <cstdio>
#include <vector>

#include "../varlen_gqa_attention_gb300/csrc/packed.cuh"

using namespace sdpa;

static int failures = 0;
#define CHECK(c)                                                \
  do {                                                          \
    if (!(c)) {                                                 \
      std::printf("FAIL %s:%d %s\n", __FILE__, __LINE__, #c);   \
      ++failures;                                               \
    }                                                           \
  } while (0)

static uint64_t state = 0x9E3779B97F4A7C15ull;
static uint64_t rnd(uint64_t n) {  // xorshift64*, below n
  state ^= state >> 12;
  state ^= state << 25;
  state ^= state >> 27;
  return (state * 0x2545F4914F6CDD1Dull >> 11) % n;
}

static void line() {
  const int nu = 1 + (int)rnd(60);
  std::vector<int64_t> base(nu), nt(nu), tw(nu);
  std::vector<int> rows(nu);
  const int64_t lead = lead_cost(kRouteSplitk, kSkQ8Few);
  int64_t Wp = 0;
  for (int u = 0; u < nu; ++u) {
    nt[u] = rnd(6) == 0 ? 0 : 1 + (int64_t)rnd(rnd(2) ? 4 : 400);
    rows[u] = 1 + (int)rnd(rnd(2) ? 8 : kSplitkRows);
    tw[u] = tile_cost(kRouteSplitk, rows[u], kSkQ8Few);
    base[u] = Wp;
    Wp += nt[u] > 0 ? lead + nt[u] * tw[u] : 0;
  }
  if (Wp == 0) return;
  const int64_t G = 1 + (int64_t)rnd(500), Gp = phase_ctas(G, Wp, kRouteSplitk, kSkQ8Few);
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
  CHECK(partial <= part_cap(nu, G, kSplitkRows));
}

int main() {
  for (int i = 0; i < 4000; ++i) line();
  // the costliest tile is what phase_ctas shares out at least
  for (int rows = 1; rows <= kSplitkRows; ++rows) CHECK(tile_cost(kRouteSplitk, rows, kSkQ8Few) <= 10);
  CHECK(phase_ctas(1000, 10 * 7 + 9, kRouteSplitk, kSkQ8Few) == 7);

  for (int i = 0; i < 100000; ++i) {
    const int Hkv = 1 + (int)rnd(9), group = 1 + (int)rnd(128), S = (int)rnd(34);
    const int64_t T = (int64_t)rnd(rnd(2) ? 300 : 9000);
    if (!sched_small_ok(T, Hkv * group, Hkv, S, kPackedTileRows)) continue;
    // the table of S segments with the most units: all but one of a row each
    int64_t units = 0, left = T;
    for (int s = 0; s < S && left > 0; ++s) {
      const int64_t n = s + 1 < S ? std::min<int64_t>(left, 1 + (int64_t)rnd(3)) : left;
      units += Hkv * ((n * group + kPackedTileRows - 1) / kPackedTileRows);
      left -= n;
    }
    CHECK(units + 31 <= kSchedThreads && S <= kSmallSegs && T <= 8192);
  }
  std::printf("failures %d\n", failures);
  return failures != 0;
}
