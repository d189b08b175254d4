"""How a pair of CTAs that gives up waits for its copies (CPU only): the function that the
kernel runs, over a model of its barriers, with every loader and the products stopping at random points
and copies landing at random times."""
import subprocess

from zero_partitioned_mixed_flat_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "loss_drain.h"

constexpr int kSlots = 3;
static std::mt19937 rng;
static int below(int n) { return (int)(rng() % (unsigned)n); }

// an mbarrier of one arrival a phase, and bytes that may be counted before they are expected
struct Barrier {
    int phases = 0, pending = 1;
    long long bytes = 0;
    void settle() {
        if (pending < 0) { std::puts("two arrivals in a phase"); std::exit(10); }
        if (pending == 0 && bytes == 0) { ++phases; pending = 1; }
    }
    void expect(uint32_t n) { bytes += n; --pending; settle(); }
    void count(uint32_t n) { bytes -= n; settle(); }
    bool done(uint32_t parity) const { return (phases & 1) != (int)parity; }
};

struct Copy { int slot; uint32_t bytes; };

struct Pair {
    Barrier full[kSlots];
    std::vector<Copy> flying;
    std::vector<uint32_t> both;                // bytes of each stage
    int placed[2] = {0, 0}, consumed = 0, finished = 0;
    uint32_t bytes[2][kSlots] = {};
    bool limited = false;

    void land() {
        const int i = below((int)flying.size());
        const Copy c = flying[i];
        flying.erase(flying.begin() + i);
        full[c.slot].count(c.bytes);
    }
    // one step of a loader, if its slot is free: the last products that used it are done
    void load(int r) {
        const int n = placed[r], slot = n % kSlots;
        if (n == (int)both.size() || n - kSlots >= finished) return;
        bytes[r][slot] = both[n];
        if (r == 0) full[slot].expect(both[n]);
        for (int k = 0; k < 4; ++k) flying.push_back({slot, both[n] / 8});   // a half is four copies
        ++placed[r];
    }
    void multiply() {
        if (consumed < (int)both.size() && full[consumed % kSlots].done((uint32_t)(consumed / kSlots) & 1u))
            ++consumed;
    }
    // drain_copies' barriers: copies go on landing while it waits
    void expect(int slot, uint32_t n) { full[slot].expect(n); }
    void count(int slot, uint32_t n) { full[slot].count(n); }
    bool wait(int slot, uint32_t parity) {
        while (!full[slot].done(parity)) {
            if (flying.empty()) { limited = true; return false; }
            land();
        }
        return true;
    }
};

int main() {
    long long uneven[2] = {0, 0}, late = 0, undone = 0;
    for (int run = 0; run < 200000; ++run) {
        rng.seed(run);
        Pair p;
        p.both.resize(below(12));
        for (auto &b : p.both) b = 8u << (8 + below(3));
        // who goes on at a step; each stops for good at a random time, the products perhaps never having begun
        const int stop[3] = {below(60), below(60), below(60)}, steps = below(70);
        for (int t = 0; t < steps; ++t) {
            const int what = below(5);
            if (what < 2 && t < stop[what]) p.load(what);
            if (what == 2 && t < stop[2]) p.multiply();
            if (what == 3 && !p.flying.empty()) p.land();
            if (what == 4 && p.finished < p.consumed) ++p.finished;
        }
        p.finished = p.consumed;                // the products in flight are waited for first
        uneven[0] += p.placed[0] > p.placed[1];
        uneven[1] += p.placed[1] > p.placed[0];
        undone += !p.flying.empty();
        const int end = p.placed[0] > p.placed[1] ? p.placed[0] : p.placed[1];
        if (end > p.consumed + kSlots) return 1;
        if (!zk::drain_copies<kSlots>(p.placed, p.bytes, p.consumed, p)) { std::printf("run %d: a wait ran out\n", run); return 2; }
        if (p.limited || !p.flying.empty()) { std::printf("run %d: %zu copies on their way\n", run, p.flying.size()); return 3; }
        int phases = 0;
        for (const auto &b : p.full) {
            if (b.bytes != 0 || b.pending != 1) { std::printf("run %d: a phase is open\n", run); return 4; }
            phases += b.phases;
        }
        if (phases != end) return 5;
        late += end > p.consumed;
    }
    // the cases it is for came up
    if (uneven[0] < 10000 || uneven[1] < 10000 || undone < 10000 || late < 10000) return 6;
    // a copy that never lands: the bounded wait says so
    Pair p;
    p.both = {1024};
    p.load(0);
    p.load(1);
    p.flying.pop_back();
    if (zk::drain_copies<kSlots>(p.placed, p.bytes, p.consumed, p)) return 7;
    std::puts("ok");
    return 0;
}
"""


def test_a_pair_that_gives_up_waits_for_its_copies(tmp_path):
    src, exe = tmp_path / "drain.cpp", tmp_path / "drain"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-I", build.CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip() == "ok", (out.returncode, out.stdout)
