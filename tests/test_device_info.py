"""SM count of the current device (csrc/tc_host.cu), against a stand-in for the CUDA runtime, and the
workspaces whose sizes depend on it."""
import contextlib
import os
import subprocess

import pytest

from block_discrete_diffusion_dg_b200 import binding as B
from block_discrete_diffusion_dg_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Two devices of different sizes and one that cannot be asked.
SRC = r'''
#include <atomic>
#include <cstdio>
#include <thread>
#include <vector>
#include <cuda_runtime_api.h>
#include "tc_host.h"
static thread_local int current = 0;
static std::atomic<int> asked{0};
static const int sms[3] = {148, 132, 0};
extern "C" cudaError_t cudaGetDevice(int *dev) { *dev = current; return cudaSuccess; }
extern "C" cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int dev) {
  ++asked;
  if (a != cudaDevAttrMultiProcessorCount || dev < 0 || dev > 2 || sms[dev] == 0) return cudaErrorInvalidDevice;
  *v = sms[dev];
  return cudaSuccess;
}
// (what an object of nvcc's registers as it is loaded)
extern "C" void **__cudaRegisterFatBinary(void *) { return nullptr; }
extern "C" void __cudaRegisterFatBinaryEnd(void **) {}
extern "C" void __cudaUnregisterFatBinary(void **) {}
#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
int main() {
  std::atomic<int> wrong{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([t, &wrong] {
      for (int i = 0; i < 2000; ++i) {
        current = (t + i) & 1;
        if (dg::num_sms() != sms[current]) ++wrong;
      }
    });
  for (std::thread &t : threads) t.join();
  CHECK(wrong == 0);
  CHECK(asked >= 2 && asked <= 16);   // once per device, or per thread that asked at the same time
  current = 2;
  CHECK(dg::num_sms() == 148);
  current = 1000;                     // more devices than are remembered
  CHECK(dg::num_sms() == 148);
  current = 1;
  CHECK(dg::num_sms() == 132);
  std::puts("ok");
  return 0;
}
'''


def test_sm_count_follows_the_current_device(tmp_path):
    src = tmp_path / "sms.cpp"
    src.write_text(SRC)
    exe, obj = tmp_path / "sms", tmp_path / "tc_host.o"
    csrc = os.path.join(ROOT, "block_discrete_diffusion_dg_b200", "csrc")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run([build.nvcc(), "-std=c++17", "-I", csrc, "-I", os.path.join(ROOT, "include"), "-c",
                    os.path.join(csrc, "tc_host.cu"), "-o", str(obj)],
                   check=True, capture_output=True, text=True)
    # (the rest of the runtime is not called)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", csrc, "-I", cuda, str(src), str(obj), "-o", str(exe),
                    "-pthread", "-Wl,--unresolved-symbols=ignore-all"],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


@pytest.mark.parametrize("size,alloc", [("dg_workspace_size", "alloc_workspace"),
                                        ("dg_paged_workspace_size", "alloc_paged_workspace")])
def test_workspaces_are_sized_on_their_device(monkeypatch, size, alloc):
    current, asked = ["cuda:0"], []

    @contextlib.contextmanager
    def device(d):
        was, current[0] = current[0], str(d)
        yield
        current[0] = was

    def of_size(*_):
        asked.append(current[0])
        return 0                                          # refused: nothing is allocated

    monkeypatch.setattr(B.torch.cuda, "device", device)
    monkeypatch.setattr(B, size, of_size)
    for d in ("cuda:1", "cuda", "cpu"):
        with pytest.raises(B.DgError):
            getattr(B, alloc)(None, 1, 1, 0, device=d)
    assert asked == ["cuda:1", "cuda:0", "cuda:0"]
