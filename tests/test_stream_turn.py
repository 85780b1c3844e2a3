"""The host's turns of a stream (csrc/stream_turn.cuh): one thread at a time for a
device and stream, others not held up.  CPU only: the source is compiled with a small
program of threads."""
import os
import shutil
import subprocess

import pytest

from paged_kv_cache_122_gb300 import build

MAIN = r"""
#include "stream_turn.cuh"
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>

int main() {
    // Eight threads, two streams on each of two devices (0 and 1 name the same stream): a
    // call's two steps have to follow each other in the stream's order.
    std::vector<int> order[2][2];
    std::atomic<int> inside[2][2] = {};
    std::atomic<int> broken{0};
    std::vector<std::thread> threads;
    for (int t = 0; t < 8; ++t)
        threads.emplace_back([&, t] {
            const int dev = t & 1, st = t >> 1 & 1;
            const void *stream = st ? reinterpret_cast<const void *>(0x1000) : reinterpret_cast<const void *>(static_cast<uintptr_t>(t >> 2));
            for (int i = 0; i < 2000; ++i) {
                const pk::StreamTurn turn(dev, stream);
                if (inside[dev][st]++) ++broken;
                order[dev][st].push_back(t);
                if (i % 16 == 0) std::this_thread::yield();
                order[dev][st].push_back(t);
                --inside[dev][st];
            }
        });
    for (auto &t : threads) t.join();
    for (auto &d : order)
        for (auto &o : d) {
            if (o.size() != 8000) ++broken;
            for (size_t i = 0; i + 1 < o.size(); i += 2) broken += o[i] != o[i + 1];
        }
    // A turn of one stream holds up no other one.
    const pk::StreamTurn held(0, reinterpret_cast<const void *>(0x1000));
    std::thread other([] {
        const pk::StreamTurn a(0, nullptr), b(1, reinterpret_cast<const void *>(0x1000)), c(0, reinterpret_cast<const void *>(0x2000));
    });
    other.join();
    std::printf("broken %d\n", broken.load());
    return broken.load() != 0;
}
"""


def test_turns_of_a_stream_exclude_each_other_and_no_other_stream(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no C++ compiler")
    main = tmp_path / "main.cpp"
    main.write_text(MAIN)
    exe = tmp_path / "turns"
    shutil.copy(os.path.join(build.CSRC, "stream_turn.cpp"), tmp_path)
    subprocess.run([cxx, "-std=c++17", "-O2", "-pthread", "-I", build.CSRC, str(main), str(tmp_path / "stream_turn.cpp"), "-o",
                    str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and res.stdout == "broken 0\n"
