"""Kernels' attributes are set on every device that launches them, from any thread: the host
helper by itself, and every launcher's use of it."""
import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "adapter_sgmv_bgmv_gb300", "csrc")

PROGRAM = r"""
#include "once.h"
#include <cstdio>
#include <thread>
#include <vector>

static thread_local int current = 0;
int lora::launch_device() { return current; }

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main()
{
    // once on each device, in any order, and again where it failed
    lora::OncePerDevice once;
    int ran[80] = {}, fail = 1;
    auto go = [&](int d) {
        current = d;
        return once([&] { ++ran[d]; return fail ? cudaErrorInvalidValue : cudaSuccess; });
    };
    CHECK(go(1) == cudaErrorInvalidValue && ran[1] == 1);
    fail = 0;
    for (int d : {1, 0, 1, 63, 0, 63, 1})
        CHECK(go(d) == cudaSuccess);
    CHECK(ran[1] == 2 && ran[0] == 1 && ran[63] == 1);
    for (int i = 0; i < 3; ++i)                     // a device that has no bit: every time
        CHECK(go(70) == cudaSuccess);
    CHECK(ran[70] == 3);

    // no thread passes before the work has succeeded on its device
    for (int round = 0; round < 200; ++round) {
        lora::OncePerDevice shared;
        std::atomic<int> set[4] = {}, early{0};
        std::vector<std::thread> threads;
        for (int t = 0; t < 8; ++t)
            threads.emplace_back([&, t] {
                current = t % 4;
                shared([&] { set[t % 4].store(1); return cudaSuccess; });
                if (!set[t % 4].load())
                    ++early;
            });
        for (auto &t : threads)
            t.join();
        CHECK(early == 0);
    }
    return 0;
}
"""


def test_the_helper_runs_its_work_on_every_device(tmp_path):
    cxx = shutil.which("g++")
    home = os.path.dirname(os.path.dirname(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"))
    if cxx is None or not os.path.exists(os.path.join(home, "include", "driver_types.h")):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, "-I", os.path.join(home, "include"), str(src),
                    "-o", str(exe)], check=True, timeout=120)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout


def test_every_launcher_uses_it():
    seen = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        text = open(path).read()
        if "cudaFuncSetAttribute" in text:
            seen += 1
            assert "OncePerDevice" in text, path
        assert not re.search(r"static\s+bool\s+\w+\s*=\s*false", text), path
    assert seen == 8
