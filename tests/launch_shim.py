"""Launches of the built library as it would make them, without a GPU: a small library in the scope of a process of its own
takes the place of the HIP runtime's launch calls and notes grid, block and the kernel's first arguments. Nothing runs on a
device."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHIM = r"""
#include <stdint.h>
#include <stdio.h>
#include <string.h>
typedef struct { uint32_t x, y, z; } dims;
static dims grid_, block_;
static size_t lds_;
static void* stream_;
int noted = 4;  // of a kernel's arguments, which it has to have
int __hipPushCallConfiguration(dims grid, dims block, size_t lds, void* stream) {
  grid_ = grid, block_ = block, lds_ = lds, stream_ = stream;
  return 0;
}
int __hipPopCallConfiguration(dims* grid, dims* block, size_t* lds, void** stream) {
  *grid = grid_, *block = block_, *lds = lds_, *stream = stream_;
  return 0;
}
int hipGetLastError(void) { return 0; }
int hipLaunchKernel(const void* f, dims grid, dims block, void** args, size_t lds, void* stream) {
  (void)f, (void)lds, (void)stream;
  uint64_t a[4] = {0, 0, 0, 0};
  for (int i = 0; i < noted; ++i) memcpy(&a[i], args[i], 8);
  printf("launch %u %u %u %u %llu %llu %llu %llu\n", grid.x, grid.y, grid.z, block.x * block.y * block.z,
         (unsigned long long)a[0], (unsigned long long)a[1], (unsigned long long)a[2], (unsigned long long)a[3]);
  fflush(stdout);
  return 0;
}
"""


def build(folder):
    """That small library, compiled into ``folder``."""
    src, lib = os.path.join(folder, "shim.c"), os.path.join(folder, "shim.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", lib, src], check=True)
    return lib


class Launch:
    def __init__(self, line):
        v = [int(x) for x in line.split()[1:]]
        self.grid, self.block, self.args = v[:3], v[3], v[4:]

    @property
    def threads(self):
        return self.grid[0] * self.block


def run(lib, code, timeout=60):
    """Runs ``code`` in a process of its own, where ``lib`` is liblrmoe.so (by ctypes). Returns what it printed and the
    launches before: [(text, launches since the last text)]."""
    head = (f"import ctypes\nshim = ctypes.CDLL({lib!r}, mode=ctypes.RTLD_GLOBAL)\n"  # before the runtime: its symbols win
            "lib = ctypes.CDLL('load_recalibrated_expert_amd/liblrmoe.so')\n"
            "vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float\n"
            "def note(n): i32.in_dll(shim, 'noted').value = n\n"
            "say = lambda t: print(t, flush=True)\n")
    out = subprocess.run([sys.executable, "-c", head + code], cwd=ROOT, capture_output=True, text=True, timeout=timeout)
    assert out.returncode == 0, out.stderr[-2000:]
    found, launches = [], []
    for line in out.stdout.splitlines():
        if line.startswith("launch "):
            launches.append(Launch(line))
        else:
            found.append((line, launches))
            launches = []
    return found
