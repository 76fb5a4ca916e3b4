"""The arithmetic that cuts token ranges into chunks and parts
(csrc/token_plan.cuh), compiled for the host with signed overflow trapped: next
to the longest positions that the paged calls take, a chunk may be nearly as
long as a position. Compared with unbounded integers."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rotate_then_quantize_b200", "csrc")
MOST = 2 ** 31 - 65536          # positions lie below this

PROGRAM = r"""
#define __host__
#define __device__
#include "token_plan.cuh"
#include <cstdio>
// plan <goal> <prefix> <n> <len>...   ->  chunk, then "sequence first end" of each chunk
// parts <per> <splits> <end>          ->  "first end" of each part
int main() {
  using namespace srftq;
  char what[8];
  while (scanf("%7s", what) == 1) {
    if (what[1] == 'l') {
      int goal, prefix, n;
      static int len[4096];
      if (scanf("%d %d %d", &goal, &prefix, &n) != 3) return 1;
      int64_t total = 0;
      for (int b = 0; b < n; ++b) {
        if (scanf("%d", len + b) != 1) return 1;
        if (len[b] > prefix) total += len[b] - prefix;
      }
      const int32_t chunk = chunk_tokens(total, goal);
      printf("%d", chunk);
      for (int b = 0; b < n; ++b) {
        const int32_t k = chunks_of(len[b] > prefix ? len[b] - prefix : 0, chunk);
        for (int32_t c = 0; c < k; ++c) {
          const int32_t t0 = prefix + c * chunk;
          printf(" %d %d %d", b, t0, range_end(t0, chunk, len[b]));
        }
      }
    } else {
      int per, splits, end;
      if (scanf("%d %d %d", &per, &splits, &end) != 3) return 1;
      for (int s = 0; s < splits; ++s) printf("%d %d ", s * per, range_end(s * per, per, end));
    }
    printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined",
                    "-fsanitize-undefined-trap-on-error", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)

    def call(line):
        out = subprocess.run([str(exe)], input=line, capture_output=True, text=True, check=True)
        return [int(x) for x in out.stdout.split()]
    return call


@pytest.mark.parametrize("heads", [1, 8, 64, 1184])
@pytest.mark.parametrize("prefix,lens", [
    (0, [MOST - 1]), (0, [2147400000]), (0, [32766 * 65536]), (5, [MOST - 1, 0, 6, 5]),
    (0, [MOST - 1] * 2), (0, [MOST - 1] * 700 + [1, 0, 129]), (MOST - 200, [MOST - 1] * 300),
    (0, [1_500_000_000, 3, 0, 1_400_000_000]), (100, [0, 1, 100, 101, 228, 229, 5000]), (0, []),
    (0, [0] * 9), (0, [2048 - 17 * i for i in range(64)])])
def test_chunks_of_own_tokens(run, heads, prefix, lens):
    """The chunks cover every own token once, in order, and are no more than the
    workspace has room for."""
    goal = -(-8 * 148 // heads)
    got = run(f"plan {goal} {prefix} {len(lens)} {' '.join(map(str, lens))}\n")
    chunk, got = got[0], got[1:]
    total = sum(max(n - prefix, 0) for n in lens)
    assert chunk % 128 == 0 and 128 <= chunk < 2 ** 31
    assert chunk == min(max(-(-(-(-total // goal)) // 128) * 128, 128), 2 ** 31 - 128)
    want = [x for b, n in enumerate(lens) for t in range(prefix, n, chunk)
            for x in (b, t, min(t + chunk, n))]
    assert got == want
    assert len(got) // 3 <= goal + len(lens)


@pytest.mark.parametrize("end", [1, 63, 64, 65, 131072, 2 ** 30 + 7, MOST - 1])
@pytest.mark.parametrize("n", [1, 2, 148, 592, 2368])
def test_parts_of_a_prefix(run, end, n):
    per = -(-(-(-end // n)) // 64) * 64
    splits = -(-end // per)
    got = run(f"parts {per} {splits} {end}\n")
    assert got == [x for s in range(splits) for x in (s * per, min((s + 1) * per, end))]
    assert got[-1] == end
