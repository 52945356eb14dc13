"""What calls of the library would launch, on a machine without a GPU: the
library is loaded in a process of its own over stand-ins for the runtime's
launch functions, which note every launch and every LDS limit and run nothing.
Pointers of the calls are never followed."""

from __future__ import annotations

import functools
import json
import os
import subprocess
import sys
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = 1 << 20      # an aligned address for every pointer

STAND_INS = r"""
#include <cstdint>
#include <cstdio>
#include <map>
#include <string>
struct dim3 { uint32_t x, y, z; };
static std::map<const void*, std::string> names;
static std::string notes;
static thread_local struct { dim3 grid, block; size_t lds; void* stream; } config;
static void note(const char* what, const void* f, const std::string& rest) {
  notes += std::string(what) + " " + names[f] + " " + rest + "\n";
}
static std::string text(dim3 d) { return std::to_string(d.x) + " " + std::to_string(d.y) + " " + std::to_string(d.z); }
extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* module; return &module; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* f, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  names[f] = name;
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, void* stream) {
  config = {grid, block, lds, stream};
  return 0;
}
int __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, void** stream) {
  *grid = config.grid, *block = config.block, *lds = config.lds, *stream = config.stream;
  return 0;
}
int hipLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t lds, void*) {
  note("launch", f, text(grid) + " " + text(block) + " " + std::to_string(lds));
  return 0;
}
int hipFuncSetAttribute(const void* f, int, int value) { note("limit", f, std::to_string(value)); return 0; }
int hipGetLastError() { return 0; }
const char* launch_notes() {
  static std::string out;
  out.swap(notes);
  notes.clear();
  return out.c_str();
}
}
"""

CHILD = r"""
import ctypes, json, sys
notes = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL).launch_notes
notes.restype = ctypes.c_char_p
import mxfp8_block_scaled_06_amd as mx
lib = mx.load_library()
notes()
out = []
for fn, args in json.load(sys.stdin):
    status = getattr(lib, fn)(*args)
    out.append([status, lib.mx_last_error().decode() if status else "", notes().decode()])
json.dump(out, sys.stdout)
"""


class Launch:
    def __init__(self, line):
        _, self.kernel, *n = line.split()
        n = list(map(int, n))
        self.grid, self.block, self.lds = n[:3], n[3:6], n[6]

    @property
    def threads(self):
        """Threads along each axis."""
        return [g * b for g, b in zip(self.grid, self.block)]


class Call:
    """A call's status, error text, launches, and LDS limits [(kernel, bytes)]."""

    def __init__(self, status, text, notes):
        self.status, self.text = status, text
        lines = notes.splitlines()
        self.launches = [Launch(l) for l in lines if l.startswith("launch ")]
        self.limits = [(l.split()[1], int(l.split()[2])) for l in lines if l.startswith("limit ")]


@functools.lru_cache(maxsize=None)
def _stand_ins():
    folder = tempfile.TemporaryDirectory(prefix="mxmoe_launches_")
    src, lib = os.path.join(folder.name, "stand_ins.cpp"), os.path.join(folder.name, "stand_ins.so")
    with open(src, "w") as f:
        f.write(STAND_INS)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", src, "-o", lib], check=True)
    return folder, lib


def record(calls):
    """calls: [(entry point, arguments)] of numbers and None -> [Call]."""
    import mxfp8_block_scaled_06_amd as mx
    if not os.path.exists(mx.library_path()):
        from mxfp8_block_scaled_06_amd import build
        build.build()
    _, lib = _stand_ins()
    done = subprocess.run([sys.executable, "-c", CHILD, lib], input=json.dumps(calls), cwd=ROOT, text=True,
                          stdout=subprocess.PIPE, timeout=120)
    assert done.returncode == 0, done.returncode
    return [Call(*c) for c in json.loads(done.stdout)]
