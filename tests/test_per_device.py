"""What is worked out once a device is kept for each device, and a failure is not kept."""
import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SRC = r"""
#include <cassert>
#include <thread>
#include <vector>
#include "per_device.h"

int main() {
    static tf::PerDevice<int> t;
    int made = 0;
    auto is = [&](int v, bool ok) { return [&made, v, ok](int &x) { x = v; ++made; return ok; }; };
    assert(!t.get(1, is(5, false)) && made == 1);        // failed: asked again
    assert(*t.get(1, is(6, true)) == 6 && made == 2);
    assert(*t.get(1, is(7, false)) == 6 && made == 2);   // kept
    assert(!t.get(0, is(8, false)));                     // another device's own
    assert(*t.get(0, is(9, true)) == 9 && *t.get(1, is(1, true)) == 6);
    assert(!t.get(-1, is(1, true)) && !t.get(tf::kMaxDevices, is(1, true)));

    static tf::PerDevice<int> u;
    std::atomic<int> calls{0};
    std::vector<std::thread> all;
    for (int i = 0; i < 16; ++i)
        all.emplace_back([&, i] {
            for (int d = 0; d < 32; ++d) assert(*u.get((d + i) % 32, [&](int &x) { x = 100 + (d + i) % 32; ++calls; return true; }) == 100 + (d + i) % 32);
        });
    for (auto &x : all) x.join();
    assert(calls == 32);
    return 0;
}
"""


def test_per_device(tmp_path):
    src = tmp_path / "t.cpp"
    src.write_text(SRC)
    exe = tmp_path / "t"
    cxx = shutil.which("g++") or "g++"
    r = subprocess.run([cxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-UNDEBUG", "-I",
                        os.path.join(ROOT, "paged_mla_kv_gb300", "csrc"), str(src), "-o", str(exe), "-lpthread"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
