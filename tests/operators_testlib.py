"""A CPU build of the library's host side: csrc/kvq_abi.cpp compiled by g++ with the CUDA runtime calls and the kernel launches
replaced by recorders, so that argument checks, plans and the host mirror run without a GPU."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STUB = r"""
#include <cstring>
#include <vector>
#include <cuda_runtime.h>
#include "kvq_operators.h"
#include "kvq_reorder_plan.h"

static std::vector<int32_t> g_log;          // what the launches were given
static void put(std::initializer_list<int32_t> v) { g_log.insert(g_log.end(), v); }

extern "C" {
cudaError_t cudaMemset(void*, int, size_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 148; return cudaSuccess; }
const char* cudaGetErrorName(cudaError_t) { return "error"; }
const char* cudaGetErrorString(cudaError_t) { return "error"; }
__attribute__((visibility("default"))) int log_size() { return (int)g_log.size(); }
__attribute__((visibility("default"))) const int32_t* log_data() { return g_log.data(); }
__attribute__((visibility("default"))) void log_clear() { g_log.clear(); }
}

namespace kvq {
cudaError_t launch_append(const Geom&, unsigned char*, const void*, const void*, int, const AppendSeqs&, int, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t decode_max_ctas(const Geom&, bool, int* m) { *m = 148; return cudaSuccess; }
cudaError_t launch_decode(const Geom&, const WsLayout&, const DecodeArgs&, int, bool, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_decode_fp16(const Geom&, const WsLayout&, const DecodeArgs&, const void*, const void*, const int32_t*, int,
                               int, cudaStream_t) { return cudaSuccess; }
cudaError_t noalloc_scratch(void** p) { *p = nullptr; return cudaSuccess; }
cudaError_t launch_norm_rotary(int, int, int, const RotaryArgs&, const RotarySeqs& s, int rows, cudaStream_t) {
  put({3, s.n, s.seq0, (int32_t)s.row0, rows});
  for (int i = 0; i < s.n; ++i) put({s.row_off[i]});
  return cudaSuccess;
}
cudaError_t launch_reorder(const Geom&, unsigned char*, const ReorderMoves& m, int shared, int64_t bytes, cudaStream_t) {
  const int n = m.chain_start[m.n_chains];
  put({2, m.n_chains, n, shared, (int32_t)bytes});
  for (int i = 0; i <= m.n_chains; ++i) put({m.chain_start[i]});
  for (int i = 0; i < n; ++i) put({m.src[i], m.dst[i], m.src_was[i], m.dst_was[i], m.batch[i], m.last[i]});
  return cudaSuccess;
}
cudaError_t attend_max_ctas(const Geom&, int* m) { *m = 592; return cudaSuccess; }
cudaError_t launch_attend(const Geom&, const WsLayout& w, const AttendArgs& a, const AttendSeqs& s, bool split, cudaStream_t) {
  put({1, s.n, s.seq0, split ? 1 : 0, s.piece_off[s.n], s.unit_rows, s.slot_rows, a.residual});
  for (int i = 0; i < s.n; ++i) put({s.row_off[i], s.n_q[i], s.piece_off[i]});
  return cudaSuccess;
}
}  // namespace kvq
"""


def cuda_include():
    for cand in ("/usr/local/cuda/include", os.path.join(os.environ.get("CUDA_HOME", ""), "include")):
        if cand and os.path.exists(os.path.join(cand, "cuda_runtime.h")):
            return cand
    return None


def host_library(folder) -> ctypes.CDLL:
    gxx, inc = shutil.which("g++"), cuda_include()
    if not gxx or not inc:
        pytest.skip("g++ or the CUDA headers are not available")
    (folder / "stub.cpp").write_text(STUB)
    csrc = os.path.join(ROOT, "asymmetric_kv_cache_b200", "csrc")
    lib = folder / "libkvq_host.so"
    cmd = [gxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-I", inc, "-I", csrc, "-I", os.path.join(ROOT, "include"),
           os.path.join(csrc, "kvq_abi.cpp"), str(folder / "stub.cpp"), "-o", str(lib)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return ctypes.CDLL(str(lib))


class Host:
    """The host library with a cache handle over a buffer that nothing touches."""

    NULL, CONFIG, SMALL, CAPACITY, EMPTY, DTYPE, CUDA, ALIGN, ARG = 1, 2, 3, 4, 5, 6, 7, 8, 9
    PTR = 1 << 20          # never read

    def __init__(self, lib, kvq):
        self.lib, self.kvq = lib, kvq
        lib.kvq_last_error.restype = ctypes.c_char_p
        lib.log_data.restype = ctypes.POINTER(ctypes.c_int32)

    def cache(self, lens=(), **kw):
        k = self.kvq
        base = dict(k_bits=4, v_bits=2, group=32, head_dim=128, n_q_heads=32, n_kv_heads=8, max_seqs=8, max_tokens=4224)
        base.update(kw)
        cfg = k.make_config(**base)
        need, ws = ctypes.c_size_t(), ctypes.c_size_t()
        assert self.lib.kvq_cache_required_bytes(ctypes.byref(cfg), ctypes.byref(need), ctypes.byref(ws)) == 0
        h = ctypes.c_void_p()
        assert self.lib.kvq_cache_create(ctypes.byref(cfg), ctypes.c_void_p(self.PTR), need, ctypes.byref(h)) == 0
        self.ws = ws.value
        if lens:
            assert self.append(h, lens) == 0
        return h

    @staticmethod
    def ints(v):
        return (ctypes.c_int32 * max(1, len(v)))(*v)

    def append(self, h, n_new):
        p = ctypes.c_void_p(self.PTR)
        return self.lib.kvq_append(h, p, p, 0, self.ints(n_new), len(n_new), None)

    def lengths(self, h, n):
        out = (ctypes.c_int32 * n)()
        assert self.lib.kvq_get_lengths(h, out, n) == 0
        return list(out)

    def log(self):
        n = self.lib.log_size()
        v = list(self.lib.log_data()[:n])
        self.lib.log_clear()
        return v

    def error(self):
        return self.lib.kvq_last_error().decode()
