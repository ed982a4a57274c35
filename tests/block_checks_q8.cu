// Host-side check (built with nvcc as a host program, run by tests/test_q8_shared_blocks.py) of blocks_meet: whether two
// segments of one column write to one block of 16 store rows, against the blocks written out.
#include <cstdio>
#include <vector>

#include "../varlen_gqa_attention_gb300/csrc/packed.cuh"

using namespace sdpa;

static uint64_t state = 0x9E3779B97F4A7C15ull;
static uint64_t rnd(uint64_t n) {  // xorshift64*, below n
  state ^= state >> 12;
  state ^= state << 25;
  state ^= state >> 27;
  return (state * 0x2545F4914F6CDD1Dull >> 11) % n;
}

static std::vector<bool> blocks(int len, int end, int64_t rows) {
  std::vector<bool> b(rows / kPackedRows);
  for (int64_t p = end > len ? end - len : 0; p < end; ++p) b[p % rows / kPackedRows] = true;
  return b;
}

int main() {
  int failures = 0, met = 0;
  for (int n = 0; n < 200000; ++n) {
    const int64_t rows = kPackedRows * (1 + (int64_t)rnd(12));
    int len[2], end[2];
    for (int k = 0; k < 2; ++k) {
      end[k] = (int)rnd(rnd(2) ? rows + 1 : 5 * rows);
      // as a valid segment: at most the ring's rows are written
      len[k] = 1 + (int)rnd(rnd(3) ? 20 : rows);
      if (len[k] > rows) len[k] = (int)rows;
      if (end[k] <= rows && rnd(8) == 0) len[k] += (int)(3 * rows);  // rows before the sequence's beginning
    }
    const std::vector<bool> a = blocks(len[0], end[0], rows), b = blocks(len[1], end[1], rows);
    bool want = false;
    for (size_t i = 0; i < a.size(); ++i) want = want || (a[i] && b[i]);
    met += want;
    if (blocks_meet(len[0], end[0], len[1], end[1], rows) != want && ++failures <= 20)
      std::printf("FAIL (%d, %d) (%d, %d) rows %lld\n", len[0], end[0], len[1], end[1], (long long)rows);
  }
  const int32_t last = INT32_MAX;  // the last positions there are
  const int64_t rows = 2147483632;
  const bool far = blocks_meet(1, last, 1, last - 15, rows), same = blocks_meet(last, last, 1, last, rows);
  failures += far || !same || blocks_meet(last, 0, 1, 1, rows);
  std::printf("failures %d of 200003, %d met\n", failures, met);
  return failures != 0 || met < 10000;
}
