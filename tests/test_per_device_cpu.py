"""Host values that belong to a device (csrc/per_device.h) are kept for each device apart.  The header
is compiled against a stand-in for the CUDA runtime with several devices; and no source keeps such a
value once a process."""
import os
import re
import subprocess

from online_softmax_tiled_attn_gb300 import binding

CSRC = binding.build_lib.CSRC

RUNTIME = """
#pragma once
enum cudaError_t { cudaSuccess = 0, cudaErrorNoDevice = 100 };
enum cudaDeviceAttr { cudaDevAttrMultiProcessorCount = 16 };
extern thread_local int g_device;
inline cudaError_t cudaGetDevice(int* d) {
    if (g_device == -1) return cudaErrorNoDevice;
    *d = g_device;
    return cudaSuccess;
}
inline cudaError_t cudaDeviceGetAttribute(int* n, cudaDeviceAttr, int dev) {
    *n = 100 + dev;
    return cudaSuccess;
}
"""

PROGRAM = """
#include "per_device.h"
#include <cstdio>
#include <thread>
#include <vector>
thread_local int g_device = 0;
static int storage[70], made[70];
#define CHECK(x) if (!(x)) { std::printf("line %d: %s\\n", __LINE__, #x); return 1; }
int main() {
    osm::PerDevice<int*> addr;
    auto make = [](int dev) { ++made[dev]; return storage + dev; };
    for (int round = 0; round < 3; ++round)
        for (int dev : {0, 1, 5, 63}) {
            g_device = dev;
            CHECK(addr.get(make) == storage + dev);
            CHECK(made[dev] == 1);
            CHECK(osm::device_sm_count() == 100 + dev);
        }
    g_device = 66;  // past the slots: made anew
    CHECK(addr.get(make) == storage + 66 && addr.get(make) == storage + 66 && made[66] == 2);
    g_device = -1;  // no device: a failure, of which nothing stays
    CHECK(addr.get(make) == nullptr && osm::device_sm_count() == 0);
    osm::PerDevice<bool> ready;
    int calls = 0;
    auto third = [&](int) { return ++calls >= 3; };
    g_device = 2;
    CHECK(!ready.get(third) && !ready.get(third) && ready.get(third) && ready.get(third));
    CHECK(calls == 3);
    g_device = 3;
    CHECK(ready.get(third) && calls == 4);
    osm::PerDevice<int> many;
    std::vector<std::thread> threads;
    int wrong[8] = {};
    for (int i = 0; i < 8; ++i)
        threads.emplace_back([&, i] {
            for (int k = 0; k < 10000; ++k) {
                g_device = (i + k) % 64;
                wrong[i] += many.get([](int dev) { return 7 + dev; }) != 7 + g_device;
            }
        });
    for (auto& t : threads) t.join();
    for (int w : wrong) CHECK(w == 0);
    return 0;
}
"""


def test_values_of_several_devices(tmp_path):
    (tmp_path / "cuda_runtime_api.h").write_text(RUNTIME)
    (tmp_path / "main.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "main")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", f"-I{tmp_path}", f"-I{CSRC}",
                        str(tmp_path / "main.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_no_source_asks_one_device_for_all():
    """Kernel attributes, addresses of device variables and SM counts go through PerDevice (or an array
    indexed by the device), never through a flag that the process sets once."""
    for f in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, f)).read()
        for m in re.finditer(r"std::call_once\(", text):
            body = text[m.start():m.start() + 700].split("});")[0]
            assert not re.search(r"cudaFuncSetAttribute|cudaGetSymbolAddress|cudaGetDevice|"
                                 r"cudaOccupancy", body), f
