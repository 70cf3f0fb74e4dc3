"""Settings that are made once a device (csrc/per_device.h), on host threads: a
caller whose setting another thread is making waits for it, a setting that
failed is made again, and every key and device has its own."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_05_gb300", "csrc")

PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"

static int failures = 0;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); ++failures; } } while (0)

int main() {
    static sv::OncePerDevice once;
    static char keys[400];
    for (int round = 0; round < 20; ++round) {   // two keys, two devices, four threads each: slow settings
        std::atomic<int> calls{0};
        std::atomic<bool> made[2][2] = {};
        std::vector<std::thread> threads;
        for (int t = 0; t < 16; ++t)
            threads.emplace_back([&, t] {
                const int k = t & 1, dev = t >> 1 & 1;
                const int rc = once.run(keys + 2 * round + k, dev, [&] {
                    std::this_thread::sleep_for(std::chrono::milliseconds(2));
                    made[k][dev] = true;
                    ++calls;
                    return 0;
                });
                CHECK(rc == 0);
                CHECK(made[k][dev]);   // nobody goes on before the setting is there
            });
        for (auto& t : threads) t.join();
        CHECK(calls == 4);
    }
    int calls = 0;
    CHECK(once.run(keys + 399, 0, [&] { ++calls; return 7; }) == 7);
    CHECK(once.run(keys + 399, 0, [&] { ++calls; return 0; }) == 0);
    CHECK(once.run(keys + 399, 0, [&] { ++calls; return 7; }) == 0);
    CHECK(calls == 2);
    calls = 0;   // more than there are places for: still set, every time
    for (int again = 0; again < 2; ++again)
        for (int k = 60; k < 390; ++k) CHECK(once.run(keys + k, 5, [&] { ++calls; return 0; }) == 0);
    CHECK(calls >= 330);
    return failures != 0;
}
"""


def test_settings_once_a_device(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
