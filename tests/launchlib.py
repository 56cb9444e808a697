"""What a C entry point would launch, on the host: the library is loaded into a process of its own behind functions
that take the place of the HIP runtime's and note each launch instead of making it, on any machine.  Pointers
given to a call are never read.  Test infrastructure only."""
from __future__ import annotations

import ctypes
import functools
import json
import os
import subprocess
import sys
import tempfile
from typing import NamedTuple

import fp8_quantization_grouped_amd as fq

SOURCE = r"""
#include <stdint.h>
#include <string.h>
struct Dim { uint32_t x, y, z; };
struct Launch { const char* kernel; Dim grid, block; uint64_t shared; unsigned char arg[256]; };
static const void* functions[8192];
static const char* names[8192];
static int known = 0;
static Dim grid_now, block_now;
static uint64_t shared_now;
static void* stream_now;
extern "C" {
Launch launches[64];
int launched = 0;
void** __hipRegisterFatBinary(const void*) { static void* handle; return &handle; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
    if (known < 8192) { functions[known] = host; names[known++] = name; }
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
int __hipPushCallConfiguration(Dim g, Dim b, size_t shared, void* stream) {
    grid_now = g; block_now = b; shared_now = shared; stream_now = stream;
    return 0;
}
int __hipPopCallConfiguration(Dim* g, Dim* b, size_t* shared, void** stream) {
    *g = grid_now; *b = block_now; *shared = shared_now; *stream = stream_now;
    return 0;
}
int hipLaunchKernel(const void* f, Dim g, Dim b, void** args, size_t shared, void*) {
    if (launched == 64) return 1;
    Launch& l = launches[launched++];
    l.kernel = "";
    for (int i = 0; i < known; i++) if (functions[i] == f) l.kernel = names[i];
    l.grid = g; l.block = b; l.shared = shared;
    memcpy(l.arg, args[0], sizeof(l.arg));
    return 0;
}
int hipGetLastError() { return 0; }
int hipGetDevice(int* d) { *d = 0; return 0; }
int hipDeviceGetAttribute(int* v, int, int) { *v = 256; return 0; }
int hipGetSymbolAddress(void** p, const void*) { *p = nullptr; return 0; }
}
"""

CHILD = r"""
import ctypes, json, sys
C = ctypes
class Launch(C.Structure):
    _fields_ = [("kernel", C.c_char_p), ("grid", C.c_uint32 * 3), ("block", C.c_uint32 * 3), ("shared", C.c_uint64), ("arg", C.c_ubyte * 256)]
stub = C.CDLL(sys.argv[1], C.RTLD_GLOBAL)
L = C.CDLL(sys.argv[2])
of = {t._type_: t for t in (C.c_void_p, C.c_int64, C.c_int32, C.c_size_t, C.c_float)}
made, count = (Launch * 64).in_dll(stub, "launches"), C.c_int.in_dll(stub, "launched")
out = []
for name, result, types, args in json.load(sys.stdin):
    f = getattr(L, name)
    f.restype, f.argtypes = of[result], [of[t] for t in types]
    count.value = 0
    status = f(*args)
    out.append([status, [[l.kernel.decode(), list(l.grid), list(l.block), l.shared, bytes(l.arg).hex()] for l in made[:count.value]]])
print(json.dumps(out))
"""


class Launch(NamedTuple):
    kernel: str
    grid: list
    block: list
    shared: int
    arg: bytes  # the first 256 bytes from the kernel's first argument on


@functools.lru_cache(None)
def stub():
    d = tempfile.TemporaryDirectory()
    src, lib = os.path.join(d.name, "launches.cpp"), os.path.join(d.name, "launches.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", src, "-o", lib], check=True)
    return lib, d  # the folder goes with the process


def launches(*calls):
    """For each (entry point, arguments; pointers as numbers, the stream left out): its status and its launches."""
    given = []
    for name, args in calls:
        result, types = fq.SIGNATURES[name]
        args = [getattr(a, "value", a) for a in args] + [None]
        assert len(args) == len(types), name
        given.append([name, result._type_, [t._type_ for t in types], args])
    run = subprocess.run([sys.executable, "-c", CHILD, stub()[0], fq.LIB_PATH], input=json.dumps(given), capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    return [(status, [Launch(k, g, b, s, bytes.fromhex(a)) for k, g, b, s, a in made]) for status, made in json.loads(run.stdout)]
