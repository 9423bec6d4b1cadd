"""Host-side refusals of the serving operators: every call below fails a host check before any
device work, so fake addresses are never dereferenced."""
import ctypes as C

import pytest

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
