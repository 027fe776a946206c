"""The host's rules of the attention of chunks at the largest sizes that its checks let through: no
overflow, and the kernels that the sizes call for.  CPU only."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_deltanet_prefill_chunkwise_amd", "csrc")

MAIN = """
#include <limits.h>
#include "chunk_rules.h"
using namespace sgdn;
int main() {
  const int cap = (1 << 29) + 1;                           // under 2^28 rows: two tiles each at most, and two more
  if (chunk_many_parts(1024, cap) || !chunk_many_parts(1024, 3) || chunk_many_parts(8, 3)) return 1;
  if (chunk_small(INT_MAX, 3) || chunk_small(INT_MAX, cap) || chunk_small(255, 3) || !chunk_small(254, 256)) return 2;
  return 0;
}
"""


def test_rules_at_the_largest_sizes(tmp_path):
    src, exe = tmp_path / "rules.cpp", tmp_path / "rules"
    src.write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_workspace_of_the_most_rows():
    """2^28 - 1 rows of one head, as many requests or more: a tile record of 32 bytes for each request and
    each 128 rows, and the parts of 512 workgroups."""
    import ctypes
    from gated_deltanet_prefill_chunkwise_amd import build, ops
    if not os.path.exists(ops.LIB_PATH):
        build.build()
    rows = (1 << 28) - 1
    tiles = -(-rows // 128) + rows + 2
    parts = 2 * 512 * 128 * (128 + 2) * 4
    for batch in (rows, 2 ** 31 - 1):
        shape = ops.Paged(rows, batch, 1, 1, 128, 64, 100, 20, 0, 1, 1)
        need = ops.lib().sgdn_paged_chunk_workspace_bytes(ctypes.byref(shape))
        assert 0 <= need - (tiles * 32 + parts + 512 * 4 + 256) < 4 * 256
    shape = ops.Paged(rows + 1, rows, 1, 1, 128, 64, 100, 20, 0, 1, 1)
    assert ops.lib().sgdn_paged_chunk_workspace_bytes(ctypes.byref(shape)) == 0
