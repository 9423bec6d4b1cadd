"""Host-side refusals of the serving operators: every call below fails a host check before any
device work, so fake addresses are never dereferenced."""
import ctypes as C
import os
import random
import re

import pytest
import torch

import draft_tree_verification_masked_b200 as et
from draft_tree_verification_masked_b200 import _build


@pytest.fixture(scope="module")
def L():
    _build.build()
    return et.lib()


def _p(i):
    return C.c_void_p(0x100000 * i)          # addresses far apart and aligned


def _rejects(status, code, words):
    msg = et.lib().etree_last_error()
    assert status == code, (status, msg)
    assert words.encode() in msg, msg


def test_every_binding_name_is_exported(L):
    for name in et.EXPORTS:
        assert hasattr(L, name) and (name == "etree_last_error" or name in et.__all__), name


def test_page_plan_refusals(L):
    def plan(B=4, n=100, cu=_p(1), kv=_p(2), page=16, maxp=8, nump=32, held=_p(3), ring=_p(4),
             state=_p(5), bt=_p(6), held_out=_p(7), state_out=_p(8), cap=_p(9), slots=_p(10),
             ws=_p(11), wsb=256):
        return L.etree_page_plan(B, n, cu, kv, page, maxp, nump, held, ring, state, bt, held_out,
                                 state_out, cap, slots, ws, wsb, None)

    for B in (0, -1, 4097):
        _rejects(plan(B=B), -1, "B=")
    _rejects(plan(n=-1), -1, "n_tokens")
    for name in ("cu", "kv", "held", "ring", "state", "held_out", "state_out"):
        _rejects(plan(**{name: None}), -1, "NULL")
    _rejects(plan(bt=None), -1, "block_table")
    for page in (0, 8, 24, 1 << 21):
        _rejects(plan(page=page), -1, "page_size")
    _rejects(plan(maxp=0), -1, "max_pages")
    _rejects(plan(maxp=1 << 27), -1, "max_pages")
    for nump in (0, 1 << 27):
        _rejects(plan(nump=nump), -1, "num_pages")
    _rejects(plan(kv=C.c_void_p(0x200002)), -1, "misaligned")
    _rejects(plan(slots=C.c_void_p(0x200004)), -1, "misaligned")
    _rejects(plan(ws=None), -1, "workspace")
    _rejects(plan(wsb=128), -1, "workspace")
    _rejects(plan(held_out=_p(3)), -1, "aliases an input")
    _rejects(plan(state_out=_p(5)), -1, "aliases an input")
    _rejects(plan(cap=C.c_void_p(0x300000 + 12)), -1, "aliases an input")   # tail of pages_held
    _rejects(plan(slots=C.c_void_p(0x600000 + 8)), -1, "alias")            # inside the table


def test_kv_store_refusals(L):
    def store(slots=_p(1), n=3, k=_p(2), ks=256, v=_p(3), vs=256, kp=_p(4), vp=_p(5), num=100,
              hkv=2, d=128, ws=_p(6), wsb=256):
        return L.etree_kv_store(slots, n, k, ks, v, vs, kp, vp, num, hkv, d, ws, wsb, None)

    _rejects(store(d=64), -2, "head_dim")
    _rejects(store(hkv=0), -1, "hkv")
    _rejects(store(n=-1), -1, "n_tokens")
    for s in (255, 248, 260):
        _rejects(store(ks=s), -1, "stride")
        _rejects(store(vs=s), -1, "stride")
    for num in (0, 1 << 31):
        _rejects(store(num=num), -1, "num_slots")
    for name in ("slots", "k", "v", "kp", "vp"):
        _rejects(store(**{name: None}), -1, "NULL")
    _rejects(store(k=C.c_void_p(0x200008)), -1, "aligned")
    _rejects(store(slots=C.c_void_p(0x200004)), -1, "aligned")
    _rejects(store(ws=None), -1, "workspace")
    assert store(n=0, slots=None, k=None, v=None) == 0       # nothing to store: no device work


def _batch(**kw):
    f = dict(B=2, n_total=6, n_max=4, kv_len_max=100, cu_nodes=0x100000, parent=0x200000,
             tokens=0x300000, kv_len=0x400000, slot_base=0x500000, slot_cap=0x600000)
    f.update(kw)
    return et.Batch(**f)


def test_attn_diff_refusals(L):
    def attn(b=None, q=_p(20), qs=512, k=_p(21), ks=256, v=_p(22), vs=256, kc=_p(23), vc=_p(24),
             slots=1000, hq=4, hkv=2, d=128, scale=0.125, lam=_p(25), w=_p(26), eps=1e-5, osc=0.2,
             out=_p(27), lse=_p(28), ws=_p(29), wsb=1 << 30, paged=None):
        b = _batch() if b is None else b
        tail = (q, qs, k, ks, v, vs, kc, vc, slots, hq, hkv, d, scale, lam, w, eps, osc, out, lse,
                ws, wsb, None)
        if paged is not None:
            return L.etree_verify_attn_diff_paged(C.byref(b), *paged, *tail)
        return L.etree_verify_attn_diff(C.byref(b), *tail)

    _rejects(attn(b=_batch(B=0)), -1, "B=")
    _rejects(attn(b=_batch(n_max=65)), -1, "n_max")
    _rejects(attn(b=_batch(n_total=1)), -1, "n_total")
    _rejects(attn(b=_batch(parent=None)), -1, "NULL")
    _rejects(attn(d=64), -2, "head_dim")
    for hq, hkv in ((0, 1), (4, 0), (5, 2), (65, 1)):
        _rejects(attn(hq=hq, hkv=hkv, qs=65 * 128), -1, "hq=")
    for name in ("q", "k", "v", "kc", "vc", "out"):
        _rejects(attn(**{name: None}), -1, "NULL")
        _rejects(attn(**{name: C.c_void_p(0x900008)}), -1, "aligned")
    _rejects(attn(lse=C.c_void_p(0x900002)), -1, "aligned")
    _rejects(attn(lam=None), -1, "lambda")
    _rejects(attn(w=C.c_void_p(0x900008)), -1, "norm_w")
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        _rejects(attn(scale=scale), -1, "scale")
    for eps in (-1e-6, float("nan"), float("inf")):
        _rejects(attn(eps=eps), -1, "norm_eps")
    _rejects(attn(osc=float("inf")), -1, "out_scale")
    for bad in (504, 516, 0, -512, 1 << 40):
        _rejects(attn(qs=bad), -1, "q_stride")
    for bad in (248, 260):
        _rejects(attn(ks=bad), -1, "k_stride")
        _rejects(attn(vs=bad), -1, "v_stride")
    for slots in (0, 1 << 31):
        _rejects(attn(slots=slots), -1, "cache_slots")
    _rejects(attn(ws=None), -1, "workspace")
    _rejects(attn(ws=C.c_void_p(0x900080)), -1, "workspace")
    need = L.etree_attn_diff_workspace_size(C.byref(_batch()), 4, 2)
    assert need >= 256
    _rejects(attn(wsb=need - 1), -1, "workspace")
    for page in (0, 8, 24):
        _rejects(attn(paged=(_p(30), 4, page)), -1, "page_size")
    _rejects(attn(paged=(None, 4, 16)), -1, "block_table")
    _rejects(attn(paged=(_p(30), 0, 16)), -1, "max_pages")
    assert L.etree_attn_diff_workspace_size(C.byref(_batch(B=0)), 4, 2) == 0
    assert L.etree_attn_diff_workspace_size(C.byref(_batch()), 5, 2) == 0
    # a loose length bound sizes a workspace all the same
    assert L.etree_attn_diff_workspace_size(C.byref(_batch(kv_len_max=2 ** 31 - 1)), 4, 2) > 256


def test_w4_refusals(L):
    def lin(x=_p(1), xs=256, M=4, wq=_p(2), s=_p(3), z=_p(4), group=64, N=100, K=256, b=_p(5),
            out=_p(6), os=100, f32=0, ws=_p(7), wsb=1 << 30):
        return L.etree_w4_linear(x, xs, M, wq, s, z, group, N, K, b, out, os, f32, ws, wsb, None)

    for M in (-1, 65537):
        _rejects(lin(M=M), -1, "M=")
    for N in (0, (1 << 24) + 1):
        _rejects(lin(N=N, os=1 << 25), -1, "N=")
    for K in (0, 16, 250, 1 << 19):
        _rejects(lin(K=K, xs=1 << 20), -1, "K=")
    for group in (0, 16, 96, 256):
        _rejects(lin(group=group), -1, "group")
    _rejects(lin(group=128, K=320, xs=320), -1, "group")
    _rejects(lin(f32=2), -1, "out_f32")
    for name in ("x", "wq", "s", "out"):
        _rejects(lin(**{name: None}), -1, "NULL")
    for name in ("x", "wq", "s", "z"):
        _rejects(lin(**{name: C.c_void_p(0x900008)}), -1, "aligned")
    _rejects(lin(out=C.c_void_p(0x900002), f32=1), -1, "misaligned")
    _rejects(lin(out=C.c_void_p(0x900001)), -1, "misaligned")
    _rejects(lin(b=C.c_void_p(0x900001)), -1, "misaligned")
    for xs in (248, 260, 0, 1 << 40):
        _rejects(lin(xs=xs), -1, "x_stride")
    for os in (99, 0, 1 << 40):
        _rejects(lin(os=os), -1, "out_stride")
    _rejects(lin(ws=None), -1, "workspace")
    _rejects(lin(ws=C.c_void_p(0x900080)), -1, "workspace")
    need = L.etree_w4_workspace_size(4, 100, 256)
    assert need > 256
    _rejects(lin(wsb=need - 1), -1, "workspace")
    assert L.etree_w4_workspace_size(4, 0, 256) == 0 and L.etree_w4_workspace_size(4, 100, 250) == 0
    assert lin(M=0, x=None, out=None) == 0                   # no tokens: no device work


def test_every_detail_code_of_the_kernels_is_documented_and_named(L):
    """Digits in a code's name included: the header's list, the kernels' enum and the binding."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "draft_tree_verification_masked_b200", "csrc", "common.cuh")) as f:
        enum = {int(v) for _, v in re.findall(r"\b(DET_[A-Z0-9_]+)\s*=\s*(\d+)", f.read())}
    with open(os.path.join(root, "include", "etree.h")) as f:
        hdr = f.read()
    block = hdr[hdr.index("Detail codes:"):hdr.index("etree_device_status(void")]
    listed = {int(n) for n in re.findall(r"\n \*\s+(\d+)\s+[a-z0-9]", block)}
    assert len(enum) == max(enum) + 1
    assert enum == listed == set(et.DETAIL)


@pytest.mark.parametrize("hq,hkv", [(40, 8), (8, 2), (64, 1), (3, 3)])
def test_attn_diff_workspace_serves_every_smaller_batch(L, hq, hkv):
    """Keys are split only where requests are few, so a smaller batch needs partial results that a larger one
    does not: the size holds for both."""
    def size(B, n_total, n_max, kv):
        b = _batch(B=B, n_total=n_total, n_max=n_max, kv_len_max=kv)
        return L.etree_attn_diff_workspace_size(C.byref(b), hq, hkv)

    rs = random.Random(hq)
    for _ in range(300):
        B, n_max, kv = rs.choice([1, 4, 16, 64, 300, 4096]), rs.randint(1, 64), rs.choice([0, 70, 8192, 131072])
        n_total = rs.randint(max(B, B * n_max // 2), B * n_max)
        if n_total * hq > 1 << 26:
            continue
        whole = size(B, n_total, n_max, kv)
        assert 0 < whole < 1 << 30
        for _ in range(20):
            b, n, k = rs.randint(1, B), rs.randint(1, n_max), rs.randint(0, kv)
            if b <= n_total:
                nt = rs.randint(b, min(n_total, b * n))
                assert size(b, nt, n, k) <= whole, (B, n_total, n_max, kv, b, nt, n, k)


def test_w4_workspace_serves_every_smaller_product(L):
    rs = random.Random(0)
    for _ in range(2000):
        M, N, K = rs.randint(1, 300), rs.randint(1, 60000), 32 * rs.randint(1, 300)
        m, n, k = rs.randint(1, M), rs.randint(1, N), 32 * rs.randint(1, K // 32)
        assert L.etree_w4_workspace_size(m, n, k) <= L.etree_w4_workspace_size(M, N, K), (M, N, K, m, n, k)


def test_attn_diff_workspace_size_is_zero_for_batches_the_call_refuses(L):
    """More rows than a call takes: refused alike by the call and by the size."""
    b = _batch(B=4096, n_total=4096 * 64, n_max=64)
    for hq, hkv in ((512, 64), (2 ** 30, 2 ** 25), (2 ** 30, 2 ** 30)):
        assert L.etree_attn_diff_workspace_size(C.byref(b), hq, hkv) == 0
        _rejects(L.etree_verify_attn_diff(C.byref(b), _p(20), hq * 128, _p(21), hkv * 128, _p(22), hkv * 128,
                                          _p(23), _p(24), 1000, hq, hkv, 128, 0.125, _p(25), None, 0.0, 1.0,
                                          _p(27), None, _p(29), 1 << 40, None), -1, "too many rows")


def test_streams_without_the_private_shortcut(monkeypatch):
    """The current stream's handle comes from torch's public call where the raw one is not there."""
    class Stream:
        cuda_stream = 1234

    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert et._stream(None) == 1234 and et._stream(77) == 77
