"""The table of tensor maps that many key/value caches share (csrc/tmap_cache.h): the maps of every layer of a
deep model are still there when its turn comes again, and each is its own.  No GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "tmap_cache.h"
#include <cstdio>
#include <cstring>
#include <vector>
using namespace attn;
#define CHECK(c) do { if (!(c)) { std::printf("FAIL line %d: %s\n", __LINE__, #c); return 1; } } while (0)

static CUtensorMap made(int n) {
    CUtensorMap m;
    std::memset(&m, 0, sizeof m);
    std::memcpy(&m, &n, sizeof n);
    return m;
}

int main() {
    static TmapTable<512, 8> table;
    // K and V of `layers` caches, side by side in one allocation or each in its own, as allocators place them
    unsigned long long base = 0;
    for (unsigned long long step : {2ull << 20, 33554432ull, 4096ull * 1024 * 128, 512ull, 123 * 65536ull}) {
        std::vector<TmapKey> keys;
        base += 1ull << 42;
        for (int i = 0; i < 2 * 128; ++i)
            keys.push_back({0, reinterpret_cast<const void*>(base + i * step), 1, 128, 64, 4096, 64});
        CUtensorMap got;
        for (size_t i = 0; i < keys.size(); ++i)
            if (!table.lookup(keys[i], &got)) table.insert(keys[i], made((int)i));
        for (size_t i = 0; i < keys.size(); ++i) {
            CHECK(table.lookup(keys[i], &got));
            const CUtensorMap want = made((int)i);
            CHECK(std::memcmp(&got, &want, sizeof got) == 0);
        }
    }
    // every input of the encode is part of the key
    const TmapKey k{0, reinterpret_cast<const void*>(0x7e0000001000ull), 1, 128, 64, 640, 64};
    CUtensorMap got;
    CHECK(!table.lookup(k, &got));
    table.insert(k, made(7));
    TmapKey v[7] = {k, k, k, k, k, k, k};
    v[0].device = 1; v[1].ptr = reinterpret_cast<const void*>(0x7e0000002000ull); v[2].elem_bytes = 2;
    v[3].D = 64; v[4].S = 32; v[5].outer = 641; v[6].box_rows = 32;
    for (int i = 0; i < 7; ++i) CHECK(!table.lookup(v[i], &got));
    CHECK(table.lookup(k, &got));
    // many more than it holds: what is there is right, and the last one is there
    for (int i = 0; i < 20000; ++i) {
        TmapKey x = k;
        x.ptr = reinterpret_cast<const void*>(0x700000000000ull + 4096ull * i);
        table.insert(x, made(i));
        CHECK(table.lookup(x, &got));
        const CUtensorMap want = made(i);
        CHECK(std::memcmp(&got, &want, sizeof got) == 0);
    }
    std::printf("OK\n");
    return 0;
}
"""


def test_maps_of_many_caches_stay(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    inc = next((d for d in ("/usr/local/cuda/include", os.path.join(os.environ.get("CUDA_HOME", ""), "include"))
                if os.path.exists(os.path.join(d, "cuda.h"))), None)
    if inc is None:
        pytest.skip("needs cuda.h")
    src = tmp_path / "table.cpp"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", inc, "-I",
                    os.path.join(ROOT, "causal_scaled_dot_gb300", "csrc"), "-o", str(tmp_path / "table"), str(src)], check=True)
    res = subprocess.run([str(tmp_path / "table")], capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout.startswith("OK"), res.stdout
