"""Page plans and K/V stores on the GPU against their plain definitions.  Everything here is whole
numbers or bit copies, so every comparison is exact."""
import numpy as np
import pytest
import torch

import draft_tree_verification_masked_b200 as et
from oracle import serving as S

pytestmark = pytest.mark.gpu

EDEVICE, ENOSPACE = -4, -6
SENT = -77


def _ws():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


class Pool:
    """A page pool's state on the device with the oracle's copy beside it."""

    def __init__(self, B, page, max_pages, num_pages, held, seed=0, head=None):
        rs = np.random.RandomState(seed)
        self.B, self.P, self.max_pages, self.num_pages = B, page, max_pages, num_pages
        held = np.asarray(held, dtype=np.int32)
        used = int(held.sum())
        assert used <= num_pages
        ids = rs.permutation(num_pages).astype(np.int32)
        self.bt = np.full((B, max_pages), SENT, np.int32)
        self.bt[np.arange(max_pages)[None, :] < held[:, None]] = ids[:used]
        self.ring = np.full(num_pages, SENT, np.int32)
        head = int(rs.randint(0, 3 * num_pages)) if head is None else head
        self.ring[(head + np.arange(num_pages - used)) % num_pages] = ids[used:]
        self.state = np.array([head, head + num_pages - used], np.int64)
        self.held = held
        self.d_bt, self.d_ring = torch.from_numpy(self.bt).cuda(), torch.from_numpy(self.ring).cuda()
        self.d_held = [torch.from_numpy(held).cuda(), torch.empty(B, dtype=torch.int32, device="cuda")]
        self.d_state = [torch.from_numpy(self.state).cuda(),
                        torch.empty(2, dtype=torch.int64, device="cuda")]
        self.bt, self.ring = self.bt.copy(), self.ring.copy()
        self.ws = _ws()

    def call(self, kv, new, pad=0, slots=True, caps=True):
        cu = np.zeros(self.B + 1, np.int32)
        np.cumsum(new, out=cu[1:])
        nt = int(cu[-1]) + pad
        d_cu = torch.from_numpy(cu).cuda()
        d_kv = torch.from_numpy(np.asarray(kv, np.int32)).cuda()
        # a guard entry on both sides of each output
        cap = torch.full((self.B + 2,), SENT, dtype=torch.int32, device="cuda")
        slot = torch.full((nt + 2,), SENT, dtype=torch.int64, device="cuda")
        et.etree_page_plan(d_cu, d_kv, self.P, self.num_pages, self.d_held[0], self.d_ring,
                           self.d_state[0], self.d_bt, self.d_held[1], self.d_state[1],
                           cap[1:-1] if caps else None, slot[1:-1] if slots else None, self.ws)
        torch.cuda.synchronize()
        assert cap[[0, -1]].tolist() == [SENT] * 2 and slot[[0, -1]].tolist() == [SENT] * 2
        return cu, nt, cap[1:-1].cpu().numpy(), slot[1:-1].cpu().numpy()

    def step(self, kv, new, **kw):
        """One call, checked against the oracle; the state advances on both sides."""
        cu, nt, cap, slot = self.call(kv, new, **kw)
        st, held, state, o_cap, o_slot = S.page_plan(cu, kv, self.P, self.held, self.ring,
                                                     self.state, self.bt, nt)
        got = et.etree_device_status(self.ws)
        assert got == ((0, 0) if st == 0 else (ENOSPACE, 4))
        assert np.array_equal(self.d_held[1].cpu().numpy(), held)
        assert np.array_equal(self.d_state[1].cpu().numpy(), state)
        assert np.array_equal(self.d_bt.cpu().numpy(), self.bt)
        assert np.array_equal(self.d_ring.cpu().numpy(), self.ring)
        if kw.get("caps", True):
            assert np.array_equal(cap, o_cap)
        if kw.get("slots", True):
            assert np.array_equal(slot, o_slot)
        self.held, self.state = held, state
        self.d_held.reverse()
        self.d_state.reverse()
        return st


@pytest.mark.parametrize("B,page,lo,hi", [(1, 16, 1, 64), (1, 16, 1, 100000), (2, 1024, 0, 1),
                                          (33, 16, 0, 700), (257, 32, 1, 64), (1025, 64, 0, 5),
                                          (4096, 16, 0, 40)])
def test_steps_of_growing_and_finishing_requests(B, page, lo, hi):
    """Three steps: prompts from nothing; then trees, with some requests finished; then trees on
    lengths that fell short of what was reserved, so that pages come back."""
    rs = np.random.RandomState(B)
    max_pages = (hi + 200) // page + 2
    pool = Pool(B, page, max_pages, B * max_pages, np.zeros(B, np.int32), seed=B)
    new = rs.randint(lo, hi + 1, size=B)
    kv = np.zeros(B, np.int64)
    assert pool.step(kv, new) == 0
    kv, new = new.copy(), rs.randint(1, 65, size=B)
    done = rs.rand(B) < 0.2
    kv[done], new[done] = 0, 0
    assert pool.step(kv, new, pad=3) == 0
    kv = kv + np.minimum(new, rs.randint(0, 4, size=B))
    new = np.where(done, hi, rs.randint(1, 3, size=B))       # finished rows take a new prompt
    assert pool.step(kv, new, pad=70) == 0
    live = pool.held[:, None] > np.arange(max_pages)[None, :]
    ids = pool.bt[live]                                      # no page is held twice, nor free
    free = pool.ring[np.arange(*pool.state) % pool.num_pages]
    assert len(set(ids.tolist()) | set(free.tolist())) == len(ids) + len(free) == pool.num_pages


@pytest.mark.parametrize("B", [1, 7, 300])
@pytest.mark.parametrize("free", [0, 1, 10])
def test_short_pool_serves_requests_in_order(B, free):
    """The first request that does not fit and every later one that grows keep what they hold."""
    held = np.arange(B) % 3 + 1                              # each growing request takes two more
    pool = Pool(B, 16, 8, int(held.sum()) + free, held, seed=B + free)
    kv, new = held * 16, np.where(np.arange(B) % 5 == 4, 0, 17)
    st = pool.step(kv, new, pad=2)
    assert st == (ENOSPACE if (new > 0).sum() * 2 > free else 0)
    pool.step(np.zeros(B), np.zeros(B))                      # all pages come back
    assert pool.state[1] - pool.state[0] == pool.num_pages and (pool.held == 0).all()


def test_full_row_empty_batch_and_optional_outputs():
    pool = Pool(3, 16, 4, 12, [0, 0, 0], head=11)            # the ring wraps
    assert pool.step([0, 0, 0], [64, 64, 64]) == 0           # every row full, no page left
    assert pool.step([64, 64, 63], [0, 0, 1], slots=False) == 0
    assert pool.step([64, 0, 1], [0, 0, 15], caps=False) == 0
    assert pool.step([0, 0, 0], [0, 0, 0]) == 0


def test_bad_requests_are_left_as_they_are():
    held = [1, 2, 0, 3]

    def check(kv, new, expect, bad, cu_edit=None, held_edit=None):
        pool = Pool(4, 16, 4, 20, held)
        before = pool.d_bt.clone()
        if held_edit is not None:
            pool.d_held[0][bad] = held_edit
        cu = np.zeros(5, np.int32)
        np.cumsum(new, out=cu[1:])
        nt = int(cu[-1])
        if cu_edit:
            cu[cu_edit[0]] = cu_edit[1]
        slot = torch.full((nt,), SENT, dtype=torch.int64, device="cuda")
        cap = torch.full((4,), SENT, dtype=torch.int32, device="cuda")
        et.etree_page_plan(torch.from_numpy(cu).cuda(),
                           torch.tensor(kv, dtype=torch.int32, device="cuda"), 16, 20,
                           pool.d_held[0], pool.d_ring, pool.d_state[0], pool.d_bt,
                           pool.d_held[1], pool.d_state[1], cap, slot, pool.ws)
        assert et.etree_device_status(pool.ws) == (EDEVICE, expect)
        assert int(pool.d_held[1][bad]) == int(pool.d_held[0][bad])
        assert torch.equal(pool.d_bt[bad], before[bad])
        assert 0 <= int(cap[bad]) <= 64
        if cu_edit is None:
            lo = int(np.sum(new[:bad]))
            assert (slot[lo:lo + new[bad]] == -1).all()
            others = [r for r in range(4) if r != bad]
            assert (pool.d_held[1].cpu().numpy()[others] ==
                    [(kv[r] + new[r] + 15) // 16 for r in others]).all()
        return slot

    check([0, -1, 0, 0], [5, 5, 5, 5], 3, 1)
    check([0, 0, 60, 0], [5, 5, 5, 5], 3, 2)                 # more tokens than max_pages hold
    check([0, 0, 0, 0], [5, 5, 5, 5], 3, 3, held_edit=5)
    check([0, 0, 0, 0], [5, 5, 5, 5], 3, 0, held_edit=-1)
    check([0, 0, 0, 0], [5, 5, 5, 5], 2, 1, cu_edit=(2, 3))  # decreasing
    check([0, 0, 0, 0], [5, 5, 5, 5], 2, 3, cu_edit=(4, 99))  # past the slot map
    check([0, 0, 0, 0], [5, 5, 5, 5], 2, 0, cu_edit=(0, 2))
    # a page id outside the pool under a new token
    pool = Pool(2, 16, 4, 8, [2, 0])
    pool.d_bt[0, 1] = 8
    _, _, _, slot = pool.call([16, 0], [3, 3])
    assert et.etree_device_status(pool.ws) == (EDEVICE, 11)
    assert (slot[:3] == -1).all() and (slot[3:] >= 0).all()


@pytest.mark.parametrize("state", [(-1, 3), (5, 3), (0, 9)])
def test_bad_ring_state_takes_and_gives_nothing(state):
    pool = Pool(2, 16, 4, 8, [2, 0])
    pool.d_state[0].copy_(torch.tensor(state))
    ring, bt = pool.d_ring.clone(), pool.d_bt.clone()
    pool.call([0, 0], [3, 3])
    assert et.etree_device_status(pool.ws) == (EDEVICE, 14)
    assert torch.equal(pool.d_ring, ring) and torch.equal(pool.d_bt, bt)
    assert pool.d_held[1].tolist() == [2, 0] and pool.d_state[1].tolist() == list(state)


def test_ring_without_room_gives_nothing_back():
    """Two held pages come back into a ring whose state counts all pages as free."""
    pool = Pool(2, 16, 4, 8, [2, 0])
    pool.d_state[0].copy_(torch.tensor([0, 8]))
    pool.call([0, 0], [0, 0])
    assert et.etree_device_status(pool.ws) == (EDEVICE, 14)
    assert pool.d_held[1].tolist() == [2, 0] and pool.d_state[1].tolist() == [0, 8]


def test_plan_replays_from_a_graph_on_another_stream():
    """Captured on a side stream and replayed on new lengths: the same as eager calls."""
    pool = Pool(5, 16, 40, 200, [0] * 5, seed=3)
    kv = torch.zeros(5, dtype=torch.int32, device="cuda")
    cu = torch.zeros(6, dtype=torch.int32, device="cuda")
    slot = torch.empty(500, dtype=torch.int64, device="cuda")
    cap = torch.empty(5, dtype=torch.int32, device="cuda")

    def call():
        et.etree_page_plan(cu, kv, 16, 200, pool.d_held[0], pool.d_ring, pool.d_state[0],
                           pool.d_bt, pool.d_held[1], pool.d_state[1], cap, slot, pool.ws)
        pool.d_held[0].copy_(pool.d_held[1])
        pool.d_state[0].copy_(pool.d_state[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            call()
    rs = np.random.RandomState(1)
    lens = np.zeros(5, np.int64)
    for _ in range(4):
        new = rs.randint(0, 90, size=5)
        cu.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)))
        kv.copy_(torch.from_numpy(lens.astype(np.int32)))
        g.replay()
        st, held, state, o_cap, o_slot = S.page_plan(cu.tolist(), lens, 16, pool.held, pool.ring,
                                                     pool.state, pool.bt, 500)
        pool.held, pool.state = held, state
        assert np.array_equal(slot.cpu().numpy(), o_slot) and np.array_equal(cap.cpu().numpy(), o_cap)
        assert np.array_equal(pool.d_bt.cpu().numpy(), pool.bt)
        lens = lens + new
    assert et.etree_device_status(pool.ws) == (0, 0)


# ---------------------------------------------------------------------------------- K/V stores
def _bits(g, *shape):
    return torch.randint(-32768, 32767, shape, generator=g, dtype=torch.int16).view(torch.bfloat16)


@pytest.mark.parametrize("n,hkv", [(0, 2), (1, 1), (1, 8), (3, 5), (64, 3), (257, 8), (5000, 2)])
@pytest.mark.parametrize("fused", [False, True])
def test_store_moves_bits_to_their_slots_and_nowhere_else(n, hkv, fused):
    g = torch.Generator().manual_seed(n * 10 + hkv)
    slots_n = n + 50
    pools = [_bits(g, slots_n, hkv, 128) for _ in range(2)]
    slots = torch.randperm(slots_n, generator=g)[:n].contiguous()
    slots[::7] = -1
    if fused:                                                # k and v are views of one projection
        rows = _bits(g, n, 3 * hkv * 128 + 8)
        k = rows[:, 8:8 + hkv * 128].unflatten(1, (hkv, 128))
        v = rows[:, 8 + 2 * hkv * 128:].unflatten(1, (hkv, 128))
        d = rows.cuda()
        dk = d[:, 8:8 + hkv * 128].unflatten(1, (hkv, 128))
        dv = d[:, 8 + 2 * hkv * 128:].unflatten(1, (hkv, 128))
    else:
        k, v = _bits(g, n, hkv, 128), _bits(g, n, hkv, 128)
        dk, dv = k.cuda(), v.cuda()
    dp = [p.cuda() for p in pools]
    ws = _ws()
    et.etree_kv_store(slots.cuda(), dk, dv, dp[0], dp[1], ws)
    assert et.etree_device_status(ws) == (0, 0)
    for rows, pool, got in ((k, pools[0], dp[0]), (v, pools[1], dp[1])):
        want = pool.view(torch.int16).numpy().copy()
        assert S.kv_store(slots.numpy(), rows.contiguous().view(torch.int16).numpy(), want) == 0
        assert np.array_equal(got.cpu().view(torch.int16).numpy(), want)


def test_store_reports_bad_slots_and_stores_the_rest():
    g = torch.Generator().manual_seed(5)
    pool = _bits(g, 20, 2, 128)
    k = _bits(g, 5, 2, 128)
    slots = torch.tensor([3, 20, -2, -1, 19])
    dk, dv, ws = pool.cuda(), pool.cuda(), _ws()
    et.etree_kv_store(slots.cuda(), k.cuda(), k.cuda(), dk, dv, ws)
    assert et.etree_device_status(ws) == (EDEVICE, 15)
    want = pool.view(torch.int16).numpy().copy()
    assert S.kv_store(slots.numpy(), k.view(torch.int16).numpy(), want) == EDEVICE
    for got in (dk, dv):
        assert np.array_equal(got.cpu().view(torch.int16).numpy(), want)


def test_store_past_32_bit_offsets():
    """A pool of more than 2^31 elements: the last slot and one beyond 2^32 bytes."""
    hkv, slots = 8, (1 << 21) + 100
    g = torch.Generator().manual_seed(6)
    k = _bits(g, 2, hkv, 128).cuda()
    pool = torch.zeros(slots, hkv, 128, dtype=torch.bfloat16, device="cuda")
    vpool = torch.zeros_like(pool)
    at = torch.tensor([slots - 1, (1 << 20) + 3 + (1 << 20)], device="cuda")
    ws = _ws()
    et.etree_kv_store(at, k, k, pool, vpool, ws)
    assert et.etree_device_status(ws) == (0, 0)
    for p in (pool, vpool):
        assert torch.equal(p[at].view(torch.int16), k.view(torch.int16))
        assert int((p.view(torch.int16) != 0).any(-1).any(-1).sum()) == 2


@pytest.mark.parametrize("cu", [[0, 8, 2, 4, 6], [0, 5, 3, 15, 20], [0, 4, 2, 2, 9], [0, 2, 90, 5, 12],
                                [0, 3, 6, 1, 4]])
def test_a_decreasing_start_costs_other_requests_no_slot(cu):
    """Requests with a bad range keep what they hold; every token inside a valid range gets a slot, the first
    such request's where ranges overlap."""
    B, n_tokens = 4, 20
    held = [1, 2, 0, 3]
    pool = Pool(B, 16, 4, 24, held)
    kv = np.array([3, 20, 0, 40], np.int32)
    slot = torch.full((n_tokens,), SENT, dtype=torch.int64, device="cuda")
    et.etree_page_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), torch.from_numpy(kv).cuda(), 16, 24,
                       pool.d_held[0], pool.d_ring, pool.d_state[0], pool.d_bt, pool.d_held[1],
                       pool.d_state[1], None, slot, pool.ws)
    assert et.etree_device_status(pool.ws) == (EDEVICE, 2)
    bt, got = pool.d_bt.cpu().numpy(), slot.cpu().numpy()
    want = np.full(n_tokens, -1, np.int64)
    for r in reversed(range(B)):
        if 0 <= cu[r] <= cu[r + 1] <= n_tokens:
            t = kv[r] + np.arange(cu[r + 1] - cu[r])
            want[cu[r]:cu[r + 1]] = bt[r, t // 16].astype(np.int64) * 16 + t % 16
            assert int(pool.d_held[1][r]) == -(-(kv[r] + cu[r + 1] - cu[r]) // 16)
        else:
            assert int(pool.d_held[1][r]) == held[r]
    assert np.array_equal(got, want)
