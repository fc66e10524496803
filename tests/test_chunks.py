"""CPU: the chunks that a group's rows are cut into, up to the most rows a
product takes (2^31 - 129).  The rule is compiled for the host."""
import subprocess

from routed_expert_ffn_02_gb300 import _build

PROGRAM = r"""
#include <cstdio>
#include "train.cuh"
int main() {
    const long long most_rows = 2147483647LL - 128;
    long long cs[4096], n = 0;
    for (long long c = 0; c < 600; ++c) cs[n++] = c;
    for (int b = 10; b < 31; ++b)
        for (long long d = -3; d <= 3; ++d) cs[n++] = (1LL << b) + d;
    for (long long d = 0; d < 600; ++d) cs[n++] = most_rows - d;
    for (long long d = -300; d <= 300; ++d) cs[n++] = 2139127680LL + d;      // c + c / 256 passes 2^31
    for (int most : {128, 256})
        for (long long i = 0; i < n; ++i) {
            const long long c = cs[i];
            const long long size = moe::chunk_size((int)c, most), chunks = moe::chunk_count((int)c, (int)size);
            const long long want = (c + most - 1) / most;
            const bool ok = c == 0 ? size == 0 && chunks == 0
                                   : size > 0 && size <= most && size % 16 == 0 && chunks <= want &&
                                         (chunks - 1) * size < c && chunks * size >= c;
            if (!ok) {
                printf("c %lld most %d: size %lld, chunks %lld\n", c, most, size, chunks);
                return 1;
            }
        }
    puts("ok");
}
"""


def test_chunks_cover_a_group(tmp_path):
    src, exe = tmp_path / "chunks.cu", tmp_path / "chunks"
    src.write_text(PROGRAM)
    r = subprocess.run([_build.nvcc(), "-std=c++20", "-I", _build.INCLUDE, "-I", _build.CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
