"""How the blocks that share a unit of the cache attention count its pieces (csrc/cache_tickets.h), with threads
for blocks: over launches that come again with the same number, as a captured one does, some of whose blocks
fail.  No GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "cache_tickets.h"
#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>
using namespace attn;

struct Memory {
    using T = unsigned long long;
    static void pause() { if (std::rand() % 3 == 0) std::this_thread::yield(); }
    static T load(T* at) { pause(); return __atomic_load_n(at, __ATOMIC_SEQ_CST); }
    static void compare_exchange(T* at, T had, T to) {
        pause();
        __atomic_compare_exchange_n(at, &had, to, false, __ATOMIC_SEQ_CST, __ATOMIC_SEQ_CST);
    }
    static T add(T* at, T n) { pause(); return __atomic_fetch_add(at, n, __ATOMIC_SEQ_CST); }
    static void set(T* at, T bits) { pause(); __atomic_fetch_or(at, bits, __ATOMIC_SEQ_CST); }
    static void clear(T* at) { pause(); __atomic_store_n(at, 0ull, __ATOMIC_SEQ_CST); }
};

struct Unit { int first, pieces; };

int wrong = 0;

// argv[1]: 1 lets a block that failed leave without counting, as one must not.
int main(int, char** argv) {
    const bool skip = std::atoi(argv[1]) != 0;
    std::srand(11);
    for (int round = 0; round < 40; ++round) {
        // units in a row, each beginning in the block where the one before it ends
        const int most = 2 + std::rand() % 7;
        std::vector<Unit> units;
        int blocks = 1;
        for (int i = 0; i < 3; ++i) {
            const int pieces = 2 + std::rand() % (i == 1 ? 30 : 9);
            units.push_back({blocks - 1, pieces});
            blocks += pieces - 1;
        }
        std::vector<unsigned long long> tickets(2 * blocks);
        for (auto& t : tickets) t = ((unsigned long long)std::rand() << 33) ^ (unsigned long long)std::rand();
        const unsigned long long number = (unsigned long long)(round + 1) * 0x9E3779B97F4Bull << 16;
        std::vector<std::vector<std::atomic<int>>> left;  // [unit][piece]: the launch that left it last
        for (auto& u : units) left.emplace_back(u.pieces);
        for (int launch = 1; launch <= 6; ++launch) {
            std::vector<char> fails(blocks);
            const bool any = launch == 2 || launch == 4;
            if (any) for (auto& f : fails) f = std::rand() % 4 == 0;
            std::vector<std::atomic<int>> joined(units.size()), early(units.size());
            auto block = [&](int b) {
                struct Share { int unit, piece; };
                std::vector<Share> shares;
                for (size_t i = 0; i < units.size(); ++i)
                    if (b >= units[i].first && b < units[i].first + units[i].pieces) shares.push_back({(int)i, b - units[i].first});
                for (auto& s : shares) {
                    const Unit& u = units[s.unit];
                    tickets_open<Memory>(tickets.data(), blocks, number, u.first, u.pieces, s.piece, most);
                    if (!fails[b]) left[s.unit][s.piece] = launch;
                }
                if (fails[b] && skip) return;
                for (auto& s : shares) {
                    const Unit& u = units[s.unit];
                    const CacheLast last = tickets_leave<Memory>(tickets.data(), u.first, u.pieces, s.piece, most, fails[b]);
                    if (last == kMoreToCome) continue;
                    const int group = cache_group(u.pieces, most);
                    const CacheGroup g = cache_group_of(u.pieces, group, s.piece);
                    if (last == kWasLast)
                        for (int i = g.begin; i < g.begin + g.n; ++i) early[s.unit] += left[s.unit][i] != launch;
                    CacheLast all = last;
                    if (group < u.pieces) all = tickets_joined<Memory>(tickets.data(), blocks, u.first, u.pieces, most, last != kWasLast);
                    if (all != kWasLast) continue;
                    for (int i = 0; i < u.pieces; ++i) early[s.unit] += left[s.unit][i] != launch;
                    ++joined[s.unit];
                }
            };
            std::vector<std::thread> run;
            for (int b = 0; b < blocks; ++b) run.emplace_back(block, b);
            for (auto& t : run) t.join();
            for (size_t i = 0; i < units.size(); ++i) {
                bool failed = false;
                for (int b = units[i].first; b < units[i].first + units[i].pieces; ++b) failed |= fails[b] != 0;
                wrong += early[i] != 0;                    // pieces joined that this launch has not left
                wrong += joined[i] != (failed ? 0 : 1);    // once when every piece was left, else never
            }
        }
    }
    std::printf("%d wrong\n", wrong);
    return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    at = tmp_path_factory.mktemp("tickets")
    (at / "tickets.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I",
                    os.path.join(ROOT, "causal_scaled_dot_gb300", "csrc"), "-o", str(at / "tickets"), str(at / "tickets.cpp")],
                   check=True)
    return str(at / "tickets")


def run(program, skip):
    res = subprocess.run([program, str(skip)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stdout + res.stderr
    return int(res.stdout.split()[0])


def test_a_launch_after_a_failed_one_joins_its_own_pieces(program):
    assert run(program, 0) == 0


def test_a_block_that_does_not_count_is_noticed(program):
    """The same check where failed blocks leave without a count: launches after it join what was never left."""
    assert run(program, 1) > 0
