"""Kernel attributes are set on every device that a process uses, not on its first one alone.

One GPU cannot show it, so the rule's own code runs here on the CPU, with a counter in the place of
the CUDA call, and the launchers' sources are held to it."""
import os
import re
import subprocess

import pytest

from paged_kv_cache_103_gb300 import build as pa_build

PROGRAM = r"""
#include "pa_device_once.h"
#include <cassert>
#include <cstdio>
#include <thread>
#include <vector>
int main() {
    pa::DeviceOnce once;
    int calls[64] = {};
    bool works = true;
    auto set = [&](int dev) { return once(dev, [&] { ++calls[dev]; return works; }); };
    assert(set(0) && set(0) && calls[0] == 1);
    assert(set(1) && calls[1] == 1 && set(0) && set(1) && calls[0] == 1 && calls[1] == 1);
    works = false;                       // a failure is reported and tried again
    assert(!set(63) && !set(63) && calls[63] == 2);
    works = true;
    assert(set(63) && set(63) && calls[63] == 3);
    assert(!once(64, [] { return true; }) && !once(-1, [] { return true; }));
    pa::DeviceOnce other;                // a kernel's record is its own
    int n = 0;
    assert(other(0, [&] { return ++n; }) && n == 1);
    pa::DeviceOnce shared;
    std::atomic<int> bad{0};
    std::vector<std::thread> ts;
    for (int t = 0; t < 8; ++t)
        ts.emplace_back([&] {
            for (int i = 0; i < 6400; ++i)
                if (!shared(i % 64, [] { return true; })) ++bad;
        });
    for (auto& t : ts) t.join();
    assert(bad == 0);
    puts("ok");
}
"""


def test_once_on_each_device(tmp_path):
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", pa_build.CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "ok\n"


@pytest.mark.parametrize("source", pa_build.CUDA_SOURCES)
def test_attributes_are_set_per_device(source):
    """A source that sets kernel attributes keeps that per device: none of its once-per-process
    blocks does it."""
    text = open(os.path.join(pa_build.CSRC, source)).read()
    for block in re.finditer(r"std::call_once\(.*?\n    \}\);", text, re.S):
        assert "cudaFuncSetAttribute" not in block.group(0)
    if "cudaFuncSetAttribute" in text:
        assert "DeviceOnce" in text
