"""The staging ring's arithmetic, on the CPU: a region never meets one that is
still in use, whatever the order of sizes, and any size up to the buffer's has a
place."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <deque>
#include <random>
#include "span_ring.h"

struct Span { size_t off, end; int id; };

int main() {
    std::mt19937 rng(5);
    for (int round = 0; round < 400; ++round) {
        const size_t cap = size_t(256) << (rng() % 9);
        dendrite::SpanRing<int> ring;
        ring.reset(cap);
        std::deque<Span> live;   // what the device may still read, oldest first
        int waited = 0;
        for (int k = 0; k < 500; ++k) {
            const size_t bytes = 256 * (1 + rng() % (rng() % 4 ? (cap + 1023) / 1024 : cap / 256));
            size_t off = 0;
            const bool ok = ring.place(bytes, &off, [&](int id) {
                ++waited;
                if (live.empty() || live.front().id != id) { std::puts("out of order"); std::exit(1); }
                live.pop_front();
                return true;
            });
            if (!ok || off + bytes > cap || off % 256) { std::puts("no place"); return 1; }
            for (const Span& s : live)
                if (s.off < off + bytes && off < s.end) { std::puts("meets a region in use"); return 1; }
            ring.use(off, bytes, k);
            live.push_back({off, off + bytes, k});
        }
        int left = 0;
        ring.drain([&](int id) { left += id == live[left].id; });
        if (left != (int)live.size() || waited + left != 500) { std::puts("lost a region"); return 1; }
        size_t off = 1;   // a wait that fails stops there
        ring.use(0, cap, 7);
        if (ring.place(256, &off, [](int) { return false; }) || off != 1) { std::puts("went on"); return 1; }
    }
    std::puts("ok");
}
"""


def test_regions_in_use_never_meet(tmp_path):
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "copy_write_forked_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout
