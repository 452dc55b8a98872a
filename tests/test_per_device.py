"""What is done once on each device: with made-up devices and steps that fail, and by several threads."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lossless_bf16_weight_exponent_gb300", "csrc")

PROGRAM = r"""
#include <atomic>
#include <cassert>
#include <thread>
#include <vector>
#include "per_device.h"

int main()
{
    uw::OncePerDevice once;
    int runs[3] = {};
    for (int turn = 0; turn < 5; turn++)
        for (int d = 0; d < 3; d++) assert(once(d, [&] { runs[d]++; return 0; }) == 0);
    for (int d = 0; d < 3; d++) assert(runs[d] == 1);  // every device's own, not the first one's alone

    int tries = 0;  // a step that fails is tried again
    assert(once(7, [&] { tries++; return 2; }) == 2 && once(7, [&] { tries++; return 0; }) == 0 && once(7, [&] { tries++; return 0; }) == 0);
    assert(tries == 2);

    int far = 0;  // devices beyond those it keeps
    for (int turn = 0; turn < 3; turn++) assert(once(1000, [&] { far++; return 0; }) == 0 && once(-1, [&] { far++; return 0; }) == 0);
    assert(far == 6);

    uw::OncePerDevice shared;  // nobody goes on before it is done
    std::atomic<int> did[8] = {};
    std::vector<std::thread> threads;
    for (int t = 0; t < 16; t++)
        threads.emplace_back([&] {
            for (int i = 0; i < 2000; i++) {
                assert(shared(i % 8, [&] { did[i % 8]++; return 0; }) == 0);
                assert(did[i % 8] >= 1);
            }
        });
    for (auto &t : threads) t.join();
    return 0;
}
"""


def test_once_per_device(tmp_path):
    (tmp_path / "p.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, "-o", str(tmp_path / "p"), str(tmp_path / "p.cpp")], check=True)
    subprocess.run([str(tmp_path / "p")], check=True, timeout=60)
