"""The library's host code on a recorder in place of the CUDA runtime (not a test module)."""
from __future__ import annotations

import ctypes
import importlib
import os
import subprocess

import block_scaled_precision_mma_gb300 as bs

lib_build = importlib.import_module("block_scaled_precision_mma_gb300.build")

HERE = os.path.dirname(os.path.abspath(__file__))
P = 1 << 20              # an address that nothing reads
LOOKUP, LAUNCH, MALLOC, FREE = range(4)

p, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
ARGS = {
    "mx_gemm": [p, p, p, p, p, i64, i64, i64, i32, i32, i32, p],
    "mx_gemm_bias_act": [p, p, p, p, p, i32, p, i64, i64, i64, i32, i32, i32, p],
    "mx_gemm_noalloc": [p, p, p, p, p, i64, i64, i64, i32, i32, i32, p],
    "grouped_fp8_gemm": [p, p, p, p, p, p, i64, i32, i64, i64, p],
    "grouped_bf16_gemm": [p, p, p, p, i64, i32, i64, i64, p],
    "fp8_group_quantize": [p, i32, i64, i64, p, i32, p, p, p],
    "fp8_block_quantize": [p, i32, i64, i64, i64, p, p, p],
    "mx_quantize": [p, i32, i64, i64, i32, i32, p, p, p],
    "moe_plan": [p, i64, i32, i32, p, p, p, p],
    "int8_gemm": [p, p, p, p, p, p, i32, i64, i64, i64, p],
    "grouped_int8_gemm": [p, p, p, p, p, i32, p, i64, i32, i64, i64, p],
    "bsmma_reserve_workspace": [i64, p],
    "bsmma_set_int8_variant": [i32, i32],
    "bsmma_set_dense_variant": [i32],
    "bsmma_set_grouped_variant": [i32],
    "bsmma_set_grouped_tile_width": [i32],
    "bsmma_autotune_configure": [i32, ctypes.c_char_p],
}


class Event:
    def __init__(self, kind, thread, device, value, name):
        self.kind, self.thread, self.device, self.value, self.name = kind, thread, device, value, name

    def __repr__(self):
        return f"({('lookup', 'launch', 'malloc', 'free')[self.kind]} thread {self.thread} {self.name})"


def load(directory):
    """The library's objects and the recorder as one shared object."""
    bs.build()
    objects = [os.path.join(lib_build.OUT_DIR, s.replace(".cu", ".o")) for s in lib_build.SOURCES]
    if not all(map(os.path.exists, objects)):
        bs.build(force=True)
    out = os.path.join(str(directory), "libbsmma_recorded.so")
    cmd = ["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-o", out,
           os.path.join(HERE, "fake_cudart.cc")] + objects + ["-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(out)
    for name, args in ARGS.items():
        getattr(lib, name).argtypes = args
    lib.bsmma_autotune_configure(0, None)
    return lib


def events(lib):
    got = []
    thread, device, value = i32(), i32(), i64()
    name = ctypes.create_string_buffer(512)
    for i in range(lib.fake_events()):
        kind = lib.fake_event(i, ctypes.byref(thread), ctypes.byref(device), ctypes.byref(value), name, 512)
        got.append(Event(kind, thread.value, device.value, value.value, name.value.decode()))
    return got
