"""Calls in several contexts of one device: what the library remembers of one (a kernel's shared
memory limit, say) does not pass for another."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A process of its own, as the contexts are made with the driver and torch knows only the primary one.
CHILD = r"""
import ctypes as C

import numpy as np

import draft_tree_verification_masked_b200 as et

cu = C.CDLL("libcuda.so.1")


def ok(code):
    assert code == 0, code


class Arrays:
    def __init__(self):
        self.made = []

    def up(self, x):
        x = np.ascontiguousarray(x)
        p = C.c_uint64()
        ok(cu.cuMemAlloc_v2(C.byref(p), C.c_size_t(x.nbytes)))
        ok(cu.cuMemcpyHtoD_v2(p, x.ctypes.data_as(C.c_void_p), C.c_size_t(x.nbytes)))
        self.made.append(p)
        return p.value


def down(ptr, like):
    got = np.empty_like(like)
    ok(cu.cuMemcpyDtoH_v2(got.ctypes.data_as(C.c_void_p), C.c_uint64(ptr), C.c_size_t(got.nbytes)))
    return got


def bf16(rs, *shape):
    return (rs.randn(*shape).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def calls():
    L, up, rs = et.lib(), Arrays().up, np.random.RandomState(0)
    results = []
    # a 4-bit product of more than 64 tokens
    M, N, K, group = 65, 300, 512, 64
    out, size = np.zeros((M, N), np.float32), L.etree_w4_workspace_size(M, N, K)
    at, ws = up(out), up(np.zeros(size, np.uint8))
    st = L.etree_w4_linear(up(bf16(rs, M, K)), K, M, up(rs.randint(0, 256, (N, K // 2)).astype(np.uint8)),
                           up(bf16(rs, N, K // group)), None, group, N, K, None, at, N, 1, ws, size, None)
    assert st == 0, L.etree_last_error()
    assert L.etree_device_status(ws, None, None) == 0
    results.append(down(at, out))
    # differential attention of a five-node chain over 200 cached tokens
    n, kv, hq, hkv = 5, 200, 4, 2
    i32 = np.int32
    b = et.Batch(B=1, n_total=n, n_max=n, kv_len_max=kv, cu_nodes=up(np.array([0, n], i32)),
                 parent=up(np.arange(-1, n - 1, dtype=i32)), tokens=up(np.zeros(n, i32)),
                 kv_len=up(np.array([kv], i32)), slot_base=up(np.zeros(1, np.int64)),
                 slot_cap=up(np.array([kv + n], i32)))
    out, size = np.zeros((n, hq, 128), np.uint16), L.etree_attn_diff_workspace_size(C.byref(b), hq, hkv)
    at, ws = up(out), up(np.zeros(size, np.uint8))
    caches = [up(bf16(rs, kv, hkv, 128)) for _ in range(2)]
    rows = [(up(bf16(rs, n, h, 128)), h * 128) for h in (hq, hkv, hkv)]
    st = L.etree_verify_attn_diff(C.byref(b), *rows[0], *rows[1], *rows[2], *caches, kv, hq, hkv, 128,
                                  0.125, up(np.full(hq, 0.5, np.float32)), None, 0.0, 1.0, at, None,
                                  ws, size, None)
    assert st == 0, L.etree_last_error()
    assert L.etree_device_status(ws, None, None) == 0
    results.append(down(at, out))
    return results


ok(cu.cuInit(0))
first = None
for _ in range(3):
    ctx = C.c_void_p()
    ok(cu.cuCtxCreate_v2(C.byref(ctx), 0, 0))
    got = calls()
    assert all(x.any() for x in got)
    first = got if first is None else first
    assert all(np.array_equal(a, b) for a, b in zip(first, got))
print("three contexts")
"""


@pytest.mark.gpu
def test_large_shared_memory_kernels_run_in_every_context():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "three contexts" in r.stdout, r.stdout + r.stderr
