"""How many blocks the 4-bit tables' host code asks for, over a stand-in runtime whose launches go nowhere:
every valid size is launched, and nothing is divided by zero on the way.  No GPU needed."""
import os
import shutil
import subprocess

import pytest

import lm_head_vocab_gb300._lib as L
from tests.test_vocab_handle_memory import CSRC, CUDA, HERE

MAIN = r"""
#include <cstdio>
#include <vector>
#include "lmloss.h"
#include <cuda_runtime_api.h>

static std::vector<unsigned> grids;
// a launch that is not to go on
extern "C" unsigned __cudaPushCallConfiguration(dim3 grid, dim3, size_t, cudaStream_t) { return grids.push_back(grid.x), 1u; }

int main()
{
    lmloss_vocab_handle h;
    if (lmloss_vocab_create(&h, 0, 0) != LMLOSS_OK) return 1;
    for (long long D : {1, 2, 7, 8, 9, 15, 16, 31, 32, 33, 247, 248, 249, 1001, 4096, 1 << 20})
        for (long long T : {1, 5, 8, 4097, (1 << 30) - 1}) {
            lmloss_table4 t{};
            t.values = reinterpret_cast<uint8_t*>(0x10000);
            t.scales = reinterpret_cast<void*>(0x20000);
            t.ld_values = (D + 31) / 32 * 16;
            t.V = T < 100000 ? T : 100000;
            t.ld_scales = (t.V + 15) / 16 * 16;
            t.D = D;
            t.group = 32;
            for (int type : {LMLOSS_BF16, LMLOSS_FP32}) {
                lmloss_table4_lookup_args a{t, reinterpret_cast<void*>(0x30000), T, reinterpret_cast<void*>(0x40000), D, LMLOSS_INT64, type, 1.f};
                lmloss_table4_quantize_args q{t, reinterpret_cast<void*>(0x40000), D, type};
                grids.clear();
                if (lmloss_table4_lookup(h, &a, nullptr) != LMLOSS_OK) return std::printf("lookup %lld %lld\n", D, T), 2;
                if (lmloss_table4_quantize(h, &q, nullptr) != LMLOSS_OK) return std::printf("quantize %lld\n", D), 3;
                if (grids.size() < 2) return std::printf("not launched\n"), 4;
                for (unsigned g : grids)
                    if (g == 0 || g > 0x7fffffffu) return std::printf("a grid of %u at %lld columns\n", g, D), 5;
            }
        }
    return 0;
}
"""


def test_every_width_is_launched(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    main, lib, exe = (str(tmp_path / n) for n in ("main.cpp", "libunit.so", "main"))
    with open(main, "w") as f:
        f.write(MAIN)
    objs = []
    for unit in ("vocab_handle", "table4"):
        objs.append(str(tmp_path / (unit + ".o")))
        # a division by zero ends the program, on every machine
        subprocess.run([L._nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-O1", "-Xcompiler",
                        "-fPIC,-O0,-fsanitize=integer-divide-by-zero,-fsanitize-undefined-trap-on-error", "-c", "-o", objs[-1],
                        os.path.join(CSRC, unit + ".cu")], check=True)
    cxx = [cxx, "-std=c++17", "-fPIC", "-I", os.path.join(HERE, "..", "include"), "-I", os.path.join(CUDA, "include")]
    subprocess.run([*cxx, "-shared", "-Wl,-z,lazy", "-o", lib, os.path.join(HERE, "vocab_fake_runtime.cpp"), *objs], check=True)
    subprocess.run([*cxx, "-Wl,-z,lazy", "-Wl,--allow-shlib-undefined", "-o", exe, main, lib, "-Wl,-rpath," + str(tmp_path),
                    "-lpthread"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stdout + r.stderr)
