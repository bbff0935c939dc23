"""The shared-memory limit of a kernel launched with different sizes from
several threads: the limit noted is the limit set, in the order of events that
lowers it otherwise. Host code only, with a fake of the runtime's call."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SRC = r"""
#include "rb_smem.h"

#include <atomic>
#include <chrono>
#include <cstdio>
#include <initializer_list>
#include <thread>

using namespace std::chrono;

static void wait_for(const std::atomic<bool>& f) {
    const auto end = steady_clock::now() + milliseconds(300);
    while (!f && steady_clock::now() < end) std::this_thread::sleep_for(milliseconds(1));
}

int main() {
    for (int dev : {0, 3, 100}) {
        rb::SmemLimit limit;
        std::atomic<size_t> set_to{0};
        std::atomic<int> calls{0};
        std::atomic<bool> small_in{false}, large_set{false}, small_done{false};
        // the smaller size is checked first and set last, the larger one noted last
        std::thread small([&] {
            limit.raise(dev, 99328, [&](size_t b) { small_in = true; wait_for(large_set); set_to = b; ++calls; return 0; });
            small_done = true;
        });
        std::thread large([&] {
            wait_for(small_in);
            limit.raise(dev, 111616, [&](size_t b) { set_to = b; large_set = true; ++calls; wait_for(small_done); return 0; });
        });
        small.join();
        large.join();
        const auto plain = [&](size_t b) { set_to = b; ++calls; return 0; };
        limit.raise(dev, 111616, plain);
        if (set_to < 111616) return std::printf("limit %zu, 111616 needed\n", set_to.load()), 1;
        limit.raise(dev, 99328, plain);
        if (set_to < 111616) return std::printf("lowered to %zu\n", set_to.load()), 2;
        if (calls != 2) return std::printf("%d calls\n", calls.load()), 3;
        // a call that fails is reported, and made again
        if (limit.raise(dev, 200000, [&](size_t) { return 7; }) != 7) return 4;
        limit.raise(dev, 200000, plain);
        if (set_to != 200000) return 5;
        // every device has a limit of its own
        limit.raise(dev + 1, 5, plain);
        if (set_to != 5) return 6;
    }
    std::printf("ok\n");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_a_limit_is_never_lowered(tmp_path):
    src = tmp_path / "limit.cpp"
    src.write_text(SRC)
    exe = tmp_path / "limit"
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I",
                           os.path.join(ROOT, "residual_binary_weight_b200", "csrc"), str(src), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, (out.returncode, out.stdout, out.stderr)
    assert out.stdout.strip() == "ok"
