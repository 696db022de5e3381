"""What the serving calls keep for a device is kept for each device.

The CUDA runtime's calls that matter are replaced, in a child process, by a fake with several devices of
different sizes: a launch with more than 48 KB of shared memory fails unless the kernel was opted in on the
device that is current, as it does on real ones.  Nothing is launched (there may be no GPU)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(shutil.which("gcc") is None or (
    shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc")), reason="no compiler")

FAKE = r"""
#include <stddef.h>
struct dim3_ { unsigned x, y, z; };
struct config { struct dim3_ grid, block; size_t smem; void* stream; void* attrs; unsigned n; };
static int device, failures, launches, kernels;
static struct { const void* f; int dev, bytes; } opted[256];
void fake_device(int d) { device = d; }
void fake_failures(int n) { failures = n; }
int fake_launches(void) { int n = launches; launches = 0; return n; }
int cudaGetDevice(int* d) { *d = device; return 0; }
int cudaGetLastError(void) { return 0; }
int cudaDeviceGetAttribute(int* v, int a, int d) { *v = a == 16 ? 100 + d : a == 97 ? 232448 : 1 << 27; return 0; }
int cudaFuncSetAttribute(const void* f, int a, int v) {
  if (failures > 0) { --failures; return 2; }
  opted[kernels].f = f; opted[kernels].dev = device; opted[kernels++].bytes = v;
  return 0;
}
int cudaLaunchKernelExC(const struct config* c, const void* f, void** args) {
  if (c->grid.x > 0x7fffffffu || c->grid.y > 65535 || c->grid.z > 65535) return 9;
  if (c->smem > 49152) {
    int ok = 0;
    for (int i = 0; i < kernels; ++i) ok |= opted[i].f == f && opted[i].dev == device && opted[i].bytes >= (int)c->smem;
    if (!ok) return 1;
  }
  ++launches;
  return 0;
}
"""

CHILD = """
import ctypes, sys
sys.modules["torch"] = None
import weight_only_int4_quant_gb300 as tlq
lib, fake, M = tlq.load(), ctypes.CDLL(None), 1 << 20

def attention(d=128, group=128, max_q=1):
    c = tlq._KV4Cache(64 * M, 10, 4, d, 16, group)
    return lib.tl_kv4_attention(ctypes.byref(c), M, 1024, 8, 16 * M, 1024, 3 * M, 4 * M, 5 * M, 4, 2, 600, max_q, 0.1, 0,
                                512 * M, 256 * M, None)

def adapters(tokens):
    return lib.tl_lora_add(M, 256, 2 * M, 3 * M, 4 * M, 5 * M, 6 * M, 3, tokens, 4, 256, 512, 32, 2, 7 * M, 512, 12 * M,
                           512, None)

sizes = []
for device in (0, 1, 5, 0):
    fake.fake_device(device)
    for form in ((128, 128, 1), (128, 64, 8), (64, 64, 4), (128, 128, 600), (64, 64, 600)):
        st = attention(*form)
        assert st == tlq.TLQ_OK, (device, form, st, tlq.tl_last_error())
        assert fake.fake_launches() == (3 if form[2] == 600 else 2), form
    for tokens in (10, 2000):
        assert adapters(tokens) == tlq.TLQ_OK and fake.fake_launches() == 1
    sizes.append(lib.tl_kv4_attention_workspace_size(8, 4, 128, 1))
assert sizes[0] < sizes[1] < sizes[2] and sizes[3] == sizes[0], sizes  # a device has 100 + its number SMs

fake.fake_device(3)  # a failure is not remembered
fake.fake_failures(1)
assert attention() == tlq.TLQ_ECUDA
assert attention() == tlq.TLQ_OK
print("done")
"""


def run_child(code, tmp_path):
    import weight_only_int4_quant_gb300 as tlq

    tlq.build()
    (tmp_path / "fake.c").write_text(FAKE)
    so = str(tmp_path / "fake.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(tmp_path / "fake.c"), "-o", so], check=True)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT,
                       env=dict(os.environ, LD_PRELOAD=so))
    assert r.returncode == 0 and "done" in r.stdout, r.stderr


def test_shared_memory_and_sizes_by_device(tmp_path):
    run_child(CHILD, tmp_path)


MANY = """
import ctypes, sys
sys.modules["torch"] = None
import weight_only_int4_quant_gb300 as tlq
lib, fake, G = tlq.load(), ctypes.CDLL(None), 1 << 36

for n in (0, 1, 255, 257, 65535 * 256, 65535 * 256 + 1, 1 << 25, (1 << 31) - 1):
    for room in (0, 5, 1 << 30):
        st = lib.tl_kv_plan(G, 2 * G, n, 3 * G, 1, 4 * G, 32, None, 16, 100, 5 * G, 6 * G, 7 * G, 8 * G, 9 * G, room,
                            10 * G, None)
        assert st == tlq.TLQ_OK and fake.fake_launches() == 1, (n, room, st, tlq.tl_last_error())
print("done")
"""


def test_plan_of_any_number_of_requests(tmp_path):
    run_child(MANY, tmp_path)
