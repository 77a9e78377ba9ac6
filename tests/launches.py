"""The library's launches without a GPU: a process of its own loads a stand-in for the HIP runtime's launches before the
library, runs a script of calls there and reports, for each call, its status and the kernels it launched.  The
stand-in can let one launch of a call fail, as a device that is lost would."""
import json
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STAND_IN = r"""
#include <stdint.h>
#include <stdlib.h>
#include <string.h>
typedef struct { uint32_t x, y, z; } dim3;
static const void *host[65536];
static const char *name[65536];
static int kernels, launches, fails_at, last;
static dim3 grid_now, block_now;
static size_t lds_now;
static void *stream_now;
static struct { const char *name; dim3 grid, block; } seen[256];

void **__hipRegisterFatBinary(const void *data) { static void *module; return &module; }
void __hipUnregisterFatBinary(void **modules) {}
void __hipRegisterVar(void **m, void *v, char *h, char *d, int e, size_t s, int c, int g) {}
void __hipRegisterFunction(void **m, const void *f, char *d, const char *n, unsigned t, void *a, void *b, void *c, void *g, int *w) {
  if (kernels < 65536) { host[kernels] = f; name[kernels++] = strdup(n); }
}
int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, void *stream) {
  grid_now = grid; block_now = block; lds_now = lds; stream_now = stream;
  return 0;
}
int __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, void **stream) {
  *grid = grid_now; *block = block_now; *lds = lds_now; *stream = stream_now;
  return 0;
}
int hipLaunchKernel(const void *f, dim3 grid, dim3 block, void **args, size_t lds, void *stream) {
  const char *n = "?";
  for (int i = 0; i < kernels; ++i) if (host[i] == f) n = name[i];
  if (launches < 256) { seen[launches].name = n; seen[launches].grid = grid; seen[launches].block = block; }
  if (++launches != fails_at) return 0;   /* (an earlier error stays until it is asked for) */
  return last = 719;
}
int hipGetLastError(void) { int e = last; last = 0; return e; }
int hipPeekAtLastError(void) { return last; }

void stand_in_begin(int at) { launches = last = 0; fails_at = at; }
int stand_in_launches(void) { return launches; }
const char *stand_in_name(int i) { return seen[i].name; }
void stand_in_sizes(int i, uint32_t *to) { memcpy(to, &seen[i].grid, 12); memcpy(to + 3, &seen[i].block, 12); }
"""

PRELUDE = r"""
import ctypes, json, sys
sys.modules["torch"] = None   # (its HIP runtime must not come first)
sys.path.insert(0, {root!r})
hip = ctypes.CDLL({lib!r}, mode=ctypes.RTLD_GLOBAL)
hip.stand_in_name.restype = ctypes.c_char_p
from bit_vector_quantised_amd import _lib
raw = _lib.raw()
out = []
def call(fn, *args, fails_at=0):
    hip.stand_in_begin(fails_at)
    status = fn(*args)
    kernels = []
    for i in range(hip.stand_in_launches()):
        sizes = (ctypes.c_uint32 * 6)()
        hip.stand_in_sizes(i, sizes)
        kernels.append([hip.stand_in_name(i).decode(), list(sizes[:3]), list(sizes[3:])])
    out.append([status, kernels])
    return status, kernels
"""


def run(folder, script):
    """The (status, [(kernel, grid, block)]) of each call(fn, *args, fails_at=0) that the script makes."""
    lib = os.path.join(str(folder), "libstandin.so")
    source = os.path.join(str(folder), "standin.c")
    with open(source, "w") as f:
        f.write(STAND_IN)
    subprocess.run(["gcc", "-O1", "-w", "-shared", "-fPIC", "-o", lib, source], check=True)
    program = PRELUDE.format(root=ROOT, lib=lib) + script + "\nprint(json.dumps(out))\n"
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return json.loads(r.stdout.splitlines()[-1])
