"""Which kernel a product on 4-bit weights takes, and the streaming kernel's shared memory.

The plans of csrc/int4_stream.cu are host functions: compiled from the source with a small host program
(nvcc, no GPU needed, 148 SMs as on a B200).
"""
import subprocess

import pytest

from int8_mixed_precision_absmax_b200 import build as B

PROGRAM = r'''
#include "int4_stream.cu"
#include <cstdio>
bool i8mm::encode_tmap_2d(CUtensorMap*, CUtensorMapDataType, const void*, uint64_t, uint64_t, uint64_t,
                          uint32_t, uint32_t, CUtensorMapSwizzle) { return false; }
int main() {
  using namespace i8mm;
  for (int M = 1; M <= 9; ++M)
    for (int group : {32, 64, 128})
      for (int K = 32; K <= INT8MM_MAX_K; K += K < 1024 ? 32 : 992) {
        StreamPlan s = {};
        const bool fits = plan_stream(M, K, group, s);
        std::printf("%d %d %d %d %d %d %d %d %d %d %zu %d\n", M, group, K, fits, s.digits, s.warps,
                    s.per_sm, s.stages, s.xstride, s.batch, s.smem,
                    int4_stream_suits(M, 4096, K, group, 148));
      }
  const int named[][3] = {NAMED};
  for (const auto& n : named) {
    StreamPlan s = {};
    std::printf("named %d %d\n", int4_stream_suits(n[0], n[1], n[2], 128, 148),
                plan_stream(n[0], n[2], 128, s) && s.digits);
  }
  std::printf("shared %zu\n", sizeof(StreamShared));
  return 0;
}
'''

# (M, N, K): whether it streams, and in digits
NAMED = {
    (1, 4096, 4096): (1, 1), (1, 49152, 12288): (1, 1), (1, 12288, 49152): (1, 0), (1, 64, 65536): (1, 0),
    (2, 4096, 4096): (1, 0), (8, 4096, 4096): (1, 0), (3, 5120, 13824): (1, 0), (2, 270000, 32768): (1, 0),
    (1, 270000, 32768): (1, 0), (1, 560000, 16384): (1, 1), (2, 300, 65536): (0, 0), (9, 64, 1024): (0, 0)}


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("routes")
    src, exe = d / "routes.cu", d / "routes"
    src.write_text(PROGRAM.replace("NAMED", ", ".join("{%d, %d, %d}" % n for n in NAMED)))
    subprocess.check_call([B.nvcc(), *B.ARCH, "-O0", "-Xptxas", "-O0", "-std=c++17", "--expt-relaxed-constexpr",
                           "-I", B.INCLUDE, "-I", B.CSRC, str(src), "-o", str(exe)])
    return subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()


def test_routes(plans):
    got = [tuple(map(int, line.split()[1:])) for line in plans if line.startswith("named")]
    assert dict(zip(NAMED, got)) == NAMED


def test_shared_memory(plans):
    shared = int(plans[-1].split()[1])
    rows = [list(map(int, line.split())) for line in plans if line[0].isdigit()]
    assert len(rows) > 1000
    for M, group, K, fits, digits, warps, per_sm, stages, xstride, batch, smem, suits in rows:
        assert fits or not suits
        if M > 8:
            assert not fits
        if not fits:
            continue
        chunks, cols = -(-K // 256), 5 if digits else M
        assert digits in (0, M == 1)
        assert smem <= 226 * 1024 // per_sm and per_sm * (smem + 1024) <= 228 * 1024
        assert xstride % 16 == 0 and xstride >= chunks * (256 if digits else 512)
        assert stages >= 2 and batch >= 1
        # alignment, ring, activations, barriers, a scale for each chunk, two batches of partial sums
        assert smem >= (1024 + warps * stages * 4096 + cols * xstride + shared + 4 * chunks * digits
                        + 2 * batch * warps * 32 * M * 4)
