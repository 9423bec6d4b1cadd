"""Steps of one attention layer of a paged target, as a serving loop runs them: plan the pages,
project with 4-bit weights, store a prompt's rows or attend with a draft tree, project back, compact
the accepted path, and plan again.  Each stage is compared with its fp64 definition on the inputs
that the library handed it, with the tolerances of the stages' own tests."""
import numpy as np
import pytest
import torch

import draft_tree_verification_masked_b200 as et
from oracle import serving as S

pytestmark = pytest.mark.gpu

HQ, HKV, D, H, PAGE, GROUP = 8, 2, 128, 512, 16, 64
QKV = (HQ + 2 * HKV) * D


def _dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


class Weights:
    def __init__(self, n, k, seed):
        g = torch.Generator().manual_seed(seed)
        self.q = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=g)
        self.s = (0.01 * torch.randn(n, k // GROUP, generator=g)).to(torch.bfloat16)
        self.z = torch.randint(0, 16, (n, k // GROUP), dtype=torch.uint8, generator=g)
        self.dev = [x.cuda() for x in (self.q, self.s, self.z)]

    def __call__(self, x, out):
        n, k = self.q.shape[0], 2 * self.q.shape[1]
        ws = torch.zeros(et.etree_w4_workspace_size(len(x), n, k), dtype=torch.uint8, device="cuda")
        et.etree_w4_linear(x, *self.dev, GROUP, None, out, ws)
        torch.cuda.synchronize()
        xs, w = x.double().cpu().numpy(), S.w4_weights(self.q.numpy(), self.s.double().numpy(),
                                                        self.z.numpy(), GROUP)
        want, mass = xs @ w.T, np.abs(xs) @ np.abs(w).T
        tol = (128 * 2.0 ** -23 + (k / GROUP + 160) * 2.0 ** -24) * mass + 2.0 ** -8 * np.abs(want)
        assert (np.abs(out.double().cpu().numpy() - want) <= tol + 1e-30).all()


class Pool:
    """The pages of a pool and what the host knows of them."""

    def __init__(self, B, pages, max_pages):
        self.B, self.pages = B, pages
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((B, max_pages), -1, **i32)
        self.held = [torch.zeros(B, **i32), torch.zeros(B, **i32)]
        self.ring = _dev(np.random.RandomState(3).permutation(pages).astype(np.int32))
        self.state = [torch.tensor([0, pages], device="cuda"), torch.zeros_like(self.ring[:2]).long()]
        self.cap = torch.zeros(B, **i32)
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def plan(self, cu, kv, slots):
        before = [t.cpu().numpy().copy() for t in (self.held[0], self.ring, self.state[0],
                                                   self.table)]
        et.etree_page_plan(cu, kv, PAGE, self.pages, self.held[0], self.ring, self.state[0],
                           self.table, self.held[1], self.state[1], self.cap, slots, self.ws)
        assert et.etree_device_status(self.ws) == (0, 0)
        held, ring, state, table = before
        _, held_out, state_out, cap, want = S.page_plan(cu.cpu().numpy(), kv.cpu().numpy(), PAGE,
                                                        held, ring, state, table,
                                                        int(cu[-1]) if slots is None else slots.numel())
        assert np.array_equal(self.held[1].cpu().numpy(), held_out)
        assert np.array_equal(self.state[1].cpu().numpy(), state_out)
        assert np.array_equal(self.table.cpu().numpy(), table)
        assert np.array_equal(self.ring.cpu().numpy(), ring)
        assert np.array_equal(self.cap.cpu().numpy(), cap)
        if slots is not None:
            assert np.array_equal(slots.cpu().numpy(), want)
        self.held.reverse()
        self.state.reverse()


def test_prompts_then_tree_steps():
    rs, g = np.random.RandomState(0), torch.Generator().manual_seed(0)
    prompts, nodes = np.array([37, 1, 90]), np.array([6, 4, 1])
    B = len(prompts)
    pool = Pool(B, 40, 12)
    w_qkv, w_out = Weights(QKV, H, 1), Weights(H, HQ * D, 2)
    bf = torch.bfloat16
    k_pool = torch.full((pool.pages * PAGE, HKV, D), float("nan"), dtype=bf, device="cuda")
    v_pool = torch.full_like(k_pool, float("nan"))

    def views(rows):
        return (rows[:, :HQ * D].unflatten(1, (HQ, D)),
                rows[:, HQ * D:(HQ + HKV) * D].unflatten(1, (HKV, D)),
                rows[:, (HQ + HKV) * D:].unflatten(1, (HKV, D)))

    # the prompts: their pages, their projected rows, and the rows' slots
    cu = _dev(np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32))
    n = int(prompts.sum())
    slots = torch.empty(n + 2, dtype=torch.int64, device="cuda")     # a padded batch
    kv = torch.zeros(B, dtype=torch.int32, device="cuda")
    pool.plan(cu, kv, slots)
    x = torch.randn(n + 2, H, generator=g).to(bf).cuda()
    rows = torch.empty(n + 2, QKV, dtype=bf, device="cuda")
    w_qkv(x, rows)
    _, k, v = views(rows)
    et.etree_kv_store(slots, k, v, k_pool, v_pool, pool.ws)
    assert et.etree_device_status(pool.ws) == (0, 0)
    used = slots[:n]
    assert torch.equal(k_pool[used], k[:n]) and torch.equal(v_pool[used], v[:n])
    assert int(torch.isfinite(k_pool).all(2).all(1).sum()) == n      # nothing else was written
    kv = _dev(prompts.astype(np.int32))

    lam, norm_w = torch.rand(HQ, generator=g).cuda(), torch.ones(D, dtype=bf, device="cuda")
    for step in range(3):
        cu_h = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        nt = int(cu_h[-1])
        parent = np.concatenate([[-1] + [int(rs.randint(0, i)) for i in range(1, m)]
                                 for m in nodes]).astype(np.int32)
        cu = _dev(cu_h)
        pool.plan(cu, kv, None)
        x = torch.randn(nt, H, generator=g).to(bf).cuda()
        rows = torch.empty(nt, QKV, dtype=bf, device="cuda")
        w_qkv(x, rows)
        q, k, v = views(rows)
        zero = torch.zeros(nt, dtype=torch.int32, device="cuda")
        batch = et.make_batch(cu, _dev(parent), zero, kv, torch.zeros(B, dtype=torch.int64,
                                                                      device="cuda"),
                              pool.cap, int(nodes.max()), int(kv.max()))
        out = torch.empty(nt, HQ, D, dtype=bf, device="cuda")
        ws = torch.zeros(et.etree_attn_diff_workspace_size(batch, HQ, HKV), dtype=torch.uint8,
                         device="cuda")
        et.etree_verify_attn_diff_paged(batch, pool.table, PAGE, q, k, v, k_pool, v_pool, 0.125,
                                        lam, None, 0.0, 1.0, out, None, ws)
        assert et.etree_device_status(ws) == (0, 0)
        table, lens = pool.table.cpu().numpy(), kv.cpu().numpy()
        cached = [table[r, np.arange(lens[r]) // PAGE].astype(np.int64) * PAGE
                  + np.arange(lens[r]) % PAGE for r in range(B)]
        f = [t.double().cpu().numpy() for t in (q, k, v, k_pool, v_pool)]
        args = (cu_h, np.concatenate([parent]), cached)
        want, _ = S.attention_diff(*args, *f, 0.125, lam.double().cpu().numpy())
        mass, _ = S.attention_diff(*args, *f[:2], np.abs(f[2]), f[3], np.abs(f[4]), 0.125,
                                   -lam.double().cpu().numpy())
        keys = np.nanmax(np.abs(np.concatenate([f[1], f[3]])))
        Z = 0.125 * np.abs(f[0]).sum(-1).max() * keys
        tol = (2.0 ** -14 + 2 * 66 * 2.0 ** -24 * Z + 2.0 ** -18) * mass + 2.0 ** -8 * np.abs(want)
        assert (np.abs(out.double().cpu().numpy() - want) <= tol + 1e-30).all()
        y = torch.empty(nt, H, dtype=bf, device="cuda")
        w_out(out.flatten(1), y)

        # every request accepts the path to its last node
        accept, path = np.zeros(B, np.int32), np.full((B, 64), -1, np.int32)
        for r in range(B):
            chain, j = [], int(nodes[r]) - 1
            while j > 0:
                chain.append(j)
                j = int(parent[cu_h[r] + j])
            accept[r] = len(chain)
            path[r, :len(chain) + 1] = [0] + chain[::-1]
        kt, vt = k.contiguous(), v.contiguous()
        kv_out = torch.empty_like(kv)
        wsc = torch.zeros(et.etree_workspace_size(batch, HQ, HKV, D, H, 32), dtype=torch.uint8,
                          device="cuda")
        et.etree_kv_compact_paged(batch, pool.table, PAGE, _dev(accept), _dev(path), kt, vt, k_pool,
                                  v_pool, pool.pages, 1, kt.numel(), k_pool.numel(), kv_out, wsc)
        assert et.etree_device_status(wsc) == (0, 0)
        assert np.array_equal(kv_out.cpu().numpy(), lens + accept + 1)
        for r in range(B):
            kept = path[r, :accept[r] + 1].tolist()
            at = np.arange(lens[r], lens[r] + len(kept))
            slot = table[r, at // PAGE].astype(np.int64) * PAGE + at % PAGE
            assert torch.equal(k_pool[_dev(slot)], kt[cu_h[r]:][kept])
        kv = kv_out
        nodes = np.array([[3, 6, 2], [1, 1, 1], [2, 5, 6]][step])
    # the last request ends and gives its pages back
    done = kv.clone()
    done[2] = 0
    pool.plan(torch.zeros(B + 1, dtype=torch.int32, device="cuda"), done, None)
    assert int(pool.held[0][2]) == 0
