"""What libzero finds out once about a device is kept for that device only (CPU only: a
program with a cudaGetDevice of its own stands in for several devices)."""
import os
import re
import subprocess

from zero_partitioned_mixed_flat_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>

#include "per_device.h"

static thread_local int device = 0;
static cudaError_t answer = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int *dev) {
    *dev = device;
    return answer;
}

int main() {
    zk::PerDevice kept;
    int asked[70] = {};
    bool fails = true;
    auto find = [&] {
        ++asked[device];
        return fails ? -(int)cudaErrorInvalidValue : 100 + device;
    };
    // a failure is reported each time and not kept
    if (kept.get(find) != -(int)cudaErrorInvalidValue || kept.get(find) != -(int)cudaErrorInvalidValue || asked[0] != 2) return 1;
    fails = false;
    for (int round = 0; round < 3; ++round)
        for (device = 0; device < 4; ++device)
            if (kept.get(find) != 100 + device) return 2;
    if (asked[0] != 3 || asked[1] != 1 || asked[2] != 1 || asked[3] != 1) return 3;
    // a second kernel's numbers are its own
    zk::PerDevice other;
    device = 1;
    if (other.get([] { return 7; }) != 7 || kept.get(find) != 101) return 4;
    // beyond the table: found each time
    device = zk::PerDevice::kDevices;
    if (kept.get(find) != 100 + device || kept.get(find) != 100 + device || asked[device] != 2) return 5;
    answer = cudaErrorNoDevice;
    if (kept.get(find) != -(int)cudaErrorNoDevice) return 6;
    answer = cudaSuccess;
    // threads on devices of their own
    zk::PerDevice shared;
    std::vector<std::thread> threads;
    std::vector<int> wrong(16, 0);
    for (int i = 0; i < 16; ++i)
        threads.emplace_back([&, i] {
            device = i % 8;
            for (int k = 0; k < 1000; ++k) wrong[i] += shared.get([&] { return 1 + device; }) != 1 + device;
        });
    for (auto &t : threads) t.join();
    for (int n : wrong)
        if (n) return 7;
    if (zk::done_or_error(cudaSuccess) != 1 || zk::done_or_error(cudaErrorInvalidValue) != -(int)cudaErrorInvalidValue) return 8;
    std::puts("ok");
    return 0;
}
"""


def test_numbers_are_kept_for_each_device(tmp_path):
    src, exe = tmp_path / "devices.cpp", tmp_path / "devices"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-I", build.CSRC, "-I", cuda, str(src), "-o", str(exe), "-pthread"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.returncode


def test_no_source_keeps_a_devices_answer_for_the_process():
    """Attributes and occupancies of a kernel in a function's static are those of the first device."""
    for name in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for found in re.finditer(r"\bstatic const (int|cudaError_t) (\w+)\s*=", text):
            assert False, (name, found.group(0))
