"""How a release pushes its blocks: the choice that the host makes before the first launch."""
import os
import subprocess

from paged_kv_cache_233_gb300 import build as pk_build

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include "pages.h"
int main(int argc, char **argv) {
    for (int i = 1; i < argc; ++i) {
        const int n = std::atoi(argv[i]);
        for (int fits = 0; fits < 2; ++fits) {
            const int ctas = pkv::push_ctas(n, fits != 0);
            std::printf("%d %d %d\n", ctas, ctas ? pkv::push_words(n, ctas) : 0, ctas ? pkv::push_smem(n, ctas) : 0);
        }
    }
}
"""


def test_a_push_fits_or_is_refused_before_anything_runs(tmp_path):
    """One block of threads for small pools, a cluster for large ones, one again where no
    cluster has room, and none (the call is refused) where its bits would not fit either."""
    (tmp_path / "ask.cpp").write_text(SOURCE)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(pk_build._nvcc())))
    subprocess.run(["g++", "-std=c++17", "-I", pk_build.CSRC, "-I", os.path.join(cuda, "include"), "-o", str(tmp_path / "ask"),
                    str(tmp_path / "ask.cpp")], check=True)
    sizes = [1, 31, 1 << 15, (1 << 15) + 1, 1 << 20, 1_851_392, 1_851_393, 1 << 24]
    out = subprocess.run([str(tmp_path / "ask"), *map(str, sizes)], check=True, capture_output=True, text=True).stdout
    lines = [tuple(map(int, line.split())) for line in out.splitlines()]
    got = {(n, fits): lines[2 * i + fits] for i, n in enumerate(sizes) for fits in (0, 1)}
    for n in sizes:
        assert got[n, 1][0] == (1 if n <= 1 << 15 else 16)
        assert got[n, 0][0] == (1 if n <= 1_851_392 else 0)
        for fits in (0, 1):
            ctas, words, smem = got[n, fits]
            if ctas:
                assert ctas * 32 * words * 32 >= n           # a bit for every block
                assert smem == 32 * words * 4 and smem <= 226 * 1024
