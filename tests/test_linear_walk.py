"""The chunk walk of the linear-attention sweeps at the longest segments (CPU):
the function that the kernel steps with, in the kernel's loop, with the 32-bit
wrap-around that the GPU's integers have."""
import os
import shutil
import subprocess

import pytest

PROGRAM = r"""
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include "chunk_walk.h"

// the chunks left from the `skip`th on, as the kernel's loop takes them
static long walk(int begin, int len, int C, long skip) {
    long n = 0;
    for (int p0 = static_cast<int>(begin + skip * C); len > 0; p0 += C) {
        ++n;
        if (n > 1000) return -1;  // it would not end
        if (!gdn2::chunk_follows(p0, len, C)) break;
    }
    return n;
}

int main() {
    const int lens[] = {0, 1, 31, 32, 33, 63, 64, 65, 700, INT32_MAX, INT32_MAX - 1, INT32_MAX - 30, INT32_MAX - 31,
                        INT32_MAX - 32, INT32_MAX - 62, INT32_MAX - 63, INT32_MAX - 64, INT32_MAX - 65};
    int bad = 0;
    for (int C : {32, 64})
        for (int rev = 0; rev < 2; ++rev)
            for (int len : lens) {
                const int begin = rev ? -((C - len % C) % C) : 0;
                const long chunks = (static_cast<long>(len) + C - 1) / C, skip = chunks > 4 ? chunks - 4 : 0;
                const long n = walk(begin, len, C, skip);
                if (n != chunks - skip) {
                    std::printf("C=%d rev=%d len=%d: %ld chunks for %ld\n", C, rev, len, n, chunks - skip);
                    ++bad;
                }
            }
    return bad != 0;
}
"""


def test_every_walk_ends_after_its_last_chunk(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_decay_amd", "csrc")
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fwrapv", "-I", csrc, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
