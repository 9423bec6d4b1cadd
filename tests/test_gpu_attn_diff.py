"""Differential tree attention on the GPU against its fp64 definition.

Tolerances.  Each probability enters its product with V as two bf16 parts, the upper half of the
fp32 word and the upper half of what that leaves, off by less than 2^-14 of it together; the output
is rounded once (2^-8 of its value).  Scores are fp32 sums of 64 exact products, off by at most
g = 66 * 2^-24 times scale * sum |q k| (at most `Z` over a case's keys), which moves a probability
and the sum it is divided by by a factor within exp(2 g Z); exponentials, sums and divisions in
fp32 stay within 2^-18 together.  So with e = 2^-14 + 2 g Z + 2^-18,
  |d - exact| <= e (a_1 |V| + lambda a_2 |V|) =: t.
With t, the norm, whose factor f = 1 / sqrt(mean d^2 + eps) moves by at most |t| / |d| (2-norms over the
head, times 1.2 while that ratio is below 1/8), carries it to f (t + 1.2 |d| |t| / |d|_2).
"""
import numpy as np
import pytest
import torch

import draft_tree_verification_masked_b200 as et
from oracle import serving as S

pytestmark = pytest.mark.gpu

EDEVICE = -4
G_SCORE = 66 * 2.0 ** -24


class Case:
    """Inputs on the device; `cache_rows` of every request for the oracle."""

    def __init__(self, nodes, kv, hq, hkv, page=0, norm=True, fused=False, seed=0, kv_max=None,
                 lse=True, slack=64, scale=None):
        rs = np.random.RandomState(seed)
        g = torch.Generator().manual_seed(seed)
        self.nodes, self.kv, self.hq, self.hkv, self.page = nodes, kv, hq, hkv, page
        B, nt = len(nodes), int(sum(nodes))
        self.B, self.nt = B, nt
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.parent = np.concatenate(
            [[-1] + [int(rs.randint(max(0, i - 4), i)) for i in range(1, n)] for n in nodes]
        ).astype(np.int32)

        def rnd(*shape):
            return torch.randn(*shape, generator=g).to(torch.bfloat16)

        if fused:
            rows = rnd(nt, (hq + 2 * hkv) * 128 + 16)
            cut = [hq * 128, (hq + hkv) * 128, (hq + 2 * hkv) * 128]
            dev = rows.cuda()

            def views(x):
                return (x[:, :cut[0]].unflatten(1, (hq, 128)),
                        x[:, cut[0]:cut[1]].unflatten(1, (hkv, 128)),
                        x[:, cut[1]:cut[2]].unflatten(1, (hkv, 128)))
            self.host = views(rows)
            self.q, self.kt, self.vt = views(dev)
        else:
            self.host = rnd(nt, hq, 128), rnd(nt, hkv, 128), rnd(nt, hkv, 128)
            self.q, self.kt, self.vt = (x.cuda() for x in self.host)
        if page:
            maxp = (max(kv) + page - 1) // page + 2
            pages = B * maxp + 3
            self.table = rs.permutation(pages)[:B * maxp].reshape(B, maxp).astype(np.int32)
            slots = pages * page
            self.rows = [self.table[r, np.arange(kv[r]) // page].astype(np.int64) * page
                         + np.arange(kv[r]) % page for r in range(B)]
            base = np.zeros(B, np.int64)
        else:
            base = np.concatenate([[0], np.cumsum(np.asarray(kv[:-1]) + 5)]).astype(np.int64)
            slots = int(sum(kv)) + 5 * B + slack
            self.table = np.zeros((B, 1), np.int32)
            self.rows = [base[r] + np.arange(kv[r]) for r in range(B)]
        self.kc_h, self.vc_h = rnd(slots, hkv, 128), rnd(slots, hkv, 128)
        self.kc, self.vc = self.kc_h.cuda(), self.vc_h.cuda()
        self.lam_h = torch.rand(hq, generator=g) * 0.8 + 0.1
        self.w_h = (1 + 0.2 * torch.randn(128, generator=g)).to(torch.bfloat16) if norm else None
        self.eps, self.out_scale = 1e-5, 0.2 if norm else 0.7
        self.scale = 0.125 if scale is None else scale
        self.lam, self.w = self.lam_h.cuda(), self.w_h.cuda() if norm else None

        def up(x):
            return torch.from_numpy(np.ascontiguousarray(x)).cuda()
        self.dev = dict(cu=up(self.cu), parent=up(self.parent), kv=up(np.asarray(kv, np.int32)),
                        base=up(base), table=up(self.table))
        i32 = dict(dtype=torch.int32, device="cuda")
        self.batch = et.make_batch(self.dev["cu"], self.dev["parent"], torch.zeros(nt, **i32),
                                   self.dev["kv"], self.dev["base"], torch.zeros(B, **i32),
                                   max(nodes), max(kv) if kv_max is None else kv_max)
        # outputs between guard rows, the workspace between guard bytes
        self.out_g = torch.full((nt + 2, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse_g = torch.full((nt + 2, hq, 2), 7.0, device="cuda")
        self.out, self.lse = self.out_g[1:-1], self.lse_g[1:-1] if lse else None
        size = et.etree_attn_diff_workspace_size(self.batch, hq, hkv)
        self.ws_g = torch.zeros(size + 512, dtype=torch.uint8, device="cuda")
        self.ws = self.ws_g[256:-256]

    def call(self, stream=None):
        args = (self.q, self.kt, self.vt, self.kc, self.vc, self.scale, self.lam, self.w, self.eps,
                self.out_scale, self.out, self.lse, self.ws, stream)
        if self.page:
            et.etree_verify_attn_diff_paged(self.batch, self.dev["table"], self.page, *args)
        else:
            et.etree_verify_attn_diff(self.batch, *args)

    def check(self, reqs=None):
        """Outputs of the listed requests against the oracle; every guard intact."""
        torch.cuda.synchronize()
        for gt in (self.out_g, self.lse_g):
            assert (gt[0] == 7.0).all() and (gt[-1] == 7.0).all()
        assert (self.ws_g[:256] == 0).all() and (self.ws_g[-256:] == 0).all()
        f = [x.double().numpy() for x in self.host] + [self.kc_h.double().numpy(),
                                                       self.vc_h.double().numpy()]
        lam = self.lam_h.double().numpy()
        w = None if self.w_h is None else self.w_h.double().numpy()
        reqs = range(self.B) if reqs is None else reqs
        for r in reqs:
            a, b = int(self.cu[r]), int(self.cu[r + 1])
            one = (np.array([0, b - a]), self.parent[a:b], [self.rows[r]], f[0][a:b], f[1][a:b],
                   f[2][a:b], f[3], f[4], self.scale)
            d, lse = S.attention_diff(*one, lam)
            mass, _ = S.attention_diff(*one[:5], np.abs(f[2][a:b]), f[3], np.abs(f[4]), self.scale,
                                       -lam)
            G = self.hq // self.hkv
            keys = np.concatenate([f[3][self.rows[r]], f[1][a:b]])
            Z = max((np.abs(f[0][a:b, h]) @ np.abs(keys[:, h // G]).T).max()
                    for h in range(self.hq)) * self.scale
            tol = (2.0 ** -14 + 2 * G_SCORE * Z + 2.0 ** -18) * mass
            if w is not None:
                fac = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + self.eps)
                rel = np.linalg.norm(tol, axis=-1, keepdims=True) / np.linalg.norm(
                    d, axis=-1, keepdims=True)
                ok = (rel < 0.125)[..., 0]
                tol = fac * (tol + 1.2 * np.abs(d) * rel) * np.abs(w)
                d = d * fac * w
                assert ok.mean() > 0.5      # heads whose maps cancel are held to nothing
                tol[~ok] = np.inf
            d, tol = d * self.out_scale, tol * self.out_scale
            got = self.out[a:b].double().cpu().numpy()
            assert (np.abs(got - d) <= tol + 2.0 ** -8 * np.abs(d) + 1e-30).all(), r
            if self.lse is not None:
                err = np.abs(self.lse[a:b].double().cpu().numpy() - lse)
                assert (err <= 2 * G_SCORE * Z + 2.0 ** -18 + 2.0 ** -22 * np.abs(lse)).all(), r

    def run(self, reqs=None):
        self.call()
        assert et.etree_device_status(self.ws) == (0, 0)
        self.check(reqs)
        return self


@pytest.mark.parametrize("hq,hkv", [(8, 2), (5, 1), (3, 3), (64, 1), (7, 1), (40, 8)])
@pytest.mark.parametrize("page", [0, 16, 64])
def test_head_layouts_and_ragged_trees(hq, hkv, page):
    Case([5, 1, 17, 2], [70, 0, 33, 1], hq, hkv, page=page, seed=hq + page).run()


@pytest.mark.parametrize("kv", [0, 1, 15, 16, 63, 64, 65, 127, 128, 129, 321])
@pytest.mark.parametrize("page", [0, 16, 32, 128])
def test_cache_lengths_around_tiles_and_pages(kv, page):
    Case([3], [kv], 4, 2, page=page, norm=kv % 2 == 0, seed=kv).run()


@pytest.mark.parametrize("n", [1, 2, 25, 26, 51, 64])
@pytest.mark.parametrize("fused", [False, True])
def test_tree_sizes_and_strided_rows(n, fused):
    Case([n, 1], [200, 90], 5, 1, fused=fused, seed=n, lse=not fused).run()


def test_many_requests_in_dispatch_order():
    rs = np.random.RandomState(2)
    nodes, kv = rs.randint(1, 9, size=60).tolist(), rs.randint(0, 300, size=60).tolist()
    Case(nodes, kv, 2, 1, page=16, seed=1).run()
    Case(nodes, kv, 2, 1, seed=2, norm=False).run()


@pytest.mark.parametrize("page", [0, 16, 256])
def test_long_caches_split_over_many_ctas(page):
    c = Case([3, 1], [9000, 4097], 4, 2, page=page, seed=9)
    assert c.ws.numel() > 1 << 16            # partials: the plan splits the keys
    c.run()


@pytest.mark.parametrize("kv_max", [9000, 200000])
def test_a_loose_length_bound_gives_the_same_results(kv_max):
    Case([6, 2], [150, 3000], 4, 2, kv_max=kv_max, seed=4).run()


def test_large_scores_and_rising_maxima():
    """Keys whose scores grow along the cache, so that every tile moves the running maximum."""
    c = Case([4], [1500], 4, 2, seed=5, scale=0.125)
    ramp = (1 + torch.arange(c.kc_h.shape[0]) / 200.0)[:, None, None]
    c.kc_h = (c.kc_h.float() * ramp).to(torch.bfloat16)
    c.kc.copy_(c.kc_h)
    c.run()


@pytest.mark.parametrize("page", [0, 16, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -3.3e38])
def test_values_in_masked_places_do_not_reach_the_output(page, value):
    """Cache rows behind kv_len (and every unused row), other requests' nodes and unseen siblings
    hold `value` in keys and values."""
    c = Case([6, 3], [70, 31], 4, 2, page=page, seed=7)
    used = np.zeros(c.kc_h.shape[0], bool)
    for rows in c.rows:
        used[rows] = True
    for h, d in ((c.kc_h, c.kc), (c.vc_h, c.vc)):
        h[torch.from_numpy(~used)] = value
        d.copy_(h)
    # request 0: a chain 0-1-2 with leaf siblings 3, 4, 5 under the root; 4 holds `value`
    c.parent[:6] = [-1, 0, 1, 0, 0, 0]
    c.dev["parent"].copy_(torch.from_numpy(c.parent))
    keep = [t[4].clone() for t in c.host]
    for h, d in zip(c.host[1:], (c.kt, c.vt)):
        h[4] = value
        d.copy_(h)
    c.call()
    assert et.etree_device_status(c.ws) == (0, 0)
    got = c.out[4].float()
    assert abs(value) < 1e38 or not torch.isfinite(got).all()    # node 4 does see itself
    # the oracle on the same inputs; node 4's own row is compared where it is finite
    for h, k in zip(c.host[1:], keep[1:]):
        h[4] = k
    out4, lse4 = c.out[4].clone(), c.lse[4].clone()
    if abs(value) < 1e38:
        return
    c.out[4], c.lse[4] = 0, 0
    rows = [0, 1, 2, 3, 5]
    a = c.cu[0]
    f = [x.double().numpy() for x in c.host]
    d, lse = S.attention_diff(np.array([0, 6]), c.parent[:6], [c.rows[0]], f[0][:6], f[1][:6],
                              f[2][:6], c.kc_h.double().numpy(), c.vc_h.double().numpy(), c.scale,
                              c.lam_h.double().numpy(), c.w_h.double().numpy(), c.eps, c.out_scale)
    err = np.abs(c.out[:6].double().cpu().numpy() - d)[rows]
    assert err.max() <= 0.05 * np.abs(d[rows]).max()
    assert np.abs(c.lse[:6].double().cpu().numpy() - lse)[rows].max() <= 1e-4
    c.out[4], c.lse[4] = out4, lse4
    c.check([1])


def test_a_seen_infinity_reaches_exactly_its_descendants():
    """Node 1's value holds +inf in dim 3 and NaN in dim 70: rows that see node 1 are not finite
    there, the others are untouched by it (with the norm off, dims do not mix)."""
    for kv in (40, 5000):                    # one CTA, and split keys
        c = Case([6], [kv], 4, 2, norm=False, seed=8)
        c.parent[:] = [-1, 0, 1, 0, 2, 3]
        c.dev["parent"].copy_(torch.from_numpy(c.parent))
        c.call()
        torch.cuda.synchronize()
        clean = c.out.clone()
        c.vt[1, :, 3], c.vt[1, :, 70] = float("inf"), float("nan")
        c.call()
        assert et.etree_device_status(c.ws) == (0, 0)
        seen = torch.tensor([False, True, True, False, True, False], device="cuda")
        assert torch.equal(c.out[~seen], clean[~seen])
        assert not torch.isfinite(c.out[seen][..., 3]).any()
        assert torch.isnan(c.out[seen][..., 70]).all()
        keep = [i for i in range(128) if i not in (3, 70)]
        assert torch.equal(c.out[seen][..., keep], clean[seen][..., keep])


def test_invalid_requests_are_reported_and_left_alone():
    def case(**kw):
        return Case([4, 5, 3], [100, 90, 80], 4, 2, seed=11, **kw)

    c = case(kv_max=100)
    c.dev["kv"][1] = 101                     # above the declared bound
    c.call()
    assert et.etree_device_status(c.ws) == (EDEVICE, 3)
    assert (c.out[4:9] == 7.0).all()
    c.check([0, 2])
    c = case()
    c.dev["base"][2] = c.kc.shape[0] - 79    # past the pool
    c.call()
    assert et.etree_device_status(c.ws) == (EDEVICE, 3)
    assert (c.out[9:] == 7.0).all()
    c.check([0, 1])
    c = case(page=16)
    c.dev["table"][0, 2] = -1                # a used page: its keys read as zeros
    c.call()
    assert et.etree_device_status(c.ws) == (EDEVICE, 11)
    c.check([1, 2])
    c = case()
    c.dev["parent"][5] = 4                   # request 1's node 1 names a later parent
    c.call()
    assert et.etree_device_status(c.ws) == (EDEVICE, 1)
    c.check([0, 2])
    c = Case([4, 5, 3], [5000, 4000, 3000], 4, 2, seed=12)   # split keys: the merge skips it too
    c.dev["kv"][0] = -1
    c.call()
    assert et.etree_device_status(c.ws) == (EDEVICE, 3)
    assert (c.out[:4] == 7.0).all()
    c.check([1, 2])


def test_cache_rows_past_32_bit_offsets():
    """A pool of more than 2^31 elements whose request lies at its end."""
    hkv, L, slots = 8, 130, (1 << 21) + 500
    c = Case([3], [L], 16, hkv, seed=13)
    kc = torch.zeros(slots, hkv, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    kc[-L:], vc[-L:] = c.kc[:L], c.vc[:L]
    small = c.kc, c.vc
    c.kc, c.vc = kc, vc
    c.dev["base"][0] = slots - L
    c.call()
    assert et.etree_device_status(c.ws) == (0, 0)
    c.kc, c.vc = small
    c.check()


def test_replays_from_graphs_on_two_streams():
    """Two graphs with workspaces of their own replay side by side on changed inputs."""
    cs = [Case([7, 2], [700, 30], 4, 2, page=16, seed=20), Case([1], [5000], 5, 1, seed=21)]
    graphs, streams = [], [torch.cuda.Stream() for _ in cs]
    for c, s in zip(cs, streams):
        g = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            c.call()
        graphs.append(g)
    for c in cs:
        c.host[0].mul_(-1)
        c.q.mul_(-1)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c in cs:
        assert et.etree_device_status(c.ws) == (0, 0)
        c.check()


def test_equal_maps_cancel():
    """Both halves alike and lambda 1: the two maps are equal bit for bit, and so the output 0."""
    c = Case([5], [100], 4, 2, norm=False, seed=30)
    for t in (c.q, c.kt, c.kc):
        t[..., 64:] = t[..., :64]
    c.lam.fill_(1.0)
    c.call()
    torch.cuda.synchronize()
    assert (c.out == 0).all() and torch.equal(c.lse[..., 0], c.lse[..., 1])


@pytest.mark.parametrize("page", [0, 16])
def test_many_calls_give_the_same_bits(page):
    """Caches that end inside a tile, with unused rows that are not finite: the two maps of a CTA clean
    the last tiles' values together, whichever runs ahead, and the outputs wait for the last products
    of both, however short the last tile's softmax."""
    c = Case([6, 4, 1, 17] * 9, [37, 101, 230, 333] * 9, 8, 2, page=page, norm=False, seed=41)
    used = np.zeros(c.kc_h.shape[0], bool)
    for rows in c.rows:
        used[rows] = True
    for h, d in ((c.kc_h, c.kc), (c.vc_h, c.vc)):
        h[torch.from_numpy(~used)] = float("nan")
        d.copy_(h)
    c.call()
    torch.cuda.synchronize()
    assert torch.isfinite(c.out.float()).all()
    first = c.out.clone()
    for _ in range(300):
        c.call()
        assert torch.equal(c.out, first)
    c.check(range(4))


@pytest.mark.parametrize("page", [0, 16, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -3.3e38])
@pytest.mark.parametrize("kv", [[70, 31], [64, 128], [2900, 1]])
def test_values_in_masked_places_change_no_bit(page, value, kv):
    """`value` in keys and values of a leaf, of the cache rows behind kv_len and of every unused row: the rows
    that do not see it keep their bits, and every row of a clean leaf is within the derived tolerance."""
    c = Case([6, 3], kv, 4, 2, page=page, seed=7)
    c.parent[:6] = [-1, 0, 1, 0, 0, 0]       # a chain 0-1-2, and leaves 3, 4, 5 under the root
    c.dev["parent"].copy_(torch.from_numpy(c.parent))
    c.run()
    out, lse = c.out.clone(), c.lse.clone()
    used = np.zeros(c.kc_h.shape[0], bool)
    for rows in c.rows:
        used[rows] = True
    for d in (c.kc, c.vc):
        d[torch.from_numpy(~used).cuda()] = value
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    for d in (c.kt, c.vt):
        d[4] = value
    c.call()
    assert et.etree_device_status(c.ws) == (0, 0)
    keep = [i for i in range(c.nt) if i != 4]
    assert torch.equal(c.out[keep], out[keep]) and torch.equal(c.lse[keep], lse[keep])
    assert not torch.equal(c.out[4], out[4])                 # node 4 does see itself


def test_one_workspace_as_requests_finish():
    """A workspace made for the first batch serves the smaller ones after it, whose keys are split."""
    nodes, kv = [6, 3, 1, 6] * 20, [5000, 300, 4097, 2600] * 20
    ws = None
    for B in (80, 33, 5, 1):
        c = Case(nodes[:B], kv[:B], 8, 2, page=16, seed=B)
        ws = c.ws if ws is None else ws
        c.ws = ws
        c.run(range(min(B, 3)))


@pytest.mark.parametrize("kv", [[40, 90], [5000, 4000]])
@pytest.mark.parametrize("fused", [False, True])
def test_rows_behind_the_last_request_are_left_as_they_were(kv, fused):
    """A batch padded to more nodes than its requests have, its spare rows not finite, in one launch and with
    split keys."""
    c = Case([3, 4], kv, 4, 2, fused=fused, seed=50)
    c.run()
    out, lse = c.out.clone(), c.lse.clone()
    pad = 1                                  # n_total is at most B * n_max
    wide = []
    for t in (c.q, c.kt, c.vt):
        w = torch.full((c.nt + pad, t.shape[1] * 128 + 8 * fused), float("nan"), dtype=t.dtype, device="cuda")
        w = w[:, :t.shape[1] * 128].unflatten(1, (t.shape[1], 128))
        w[:c.nt] = t
        wide.append(w)
    c.q, c.kt, c.vt = wide
    i32 = dict(dtype=torch.int32, device="cuda")
    parent = torch.cat([c.dev["parent"], torch.full((pad,), -9, **i32)])
    c.batch = et.make_batch(c.dev["cu"], parent, torch.zeros(c.nt + pad, **i32), c.dev["kv"], c.dev["base"],
                            torch.zeros(2, **i32), 4, max(kv))
    c.out = torch.full((c.nt + pad, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    c.lse = torch.full((c.nt + pad, 4, 2), 7.0, device="cuda")
    c.ws = torch.zeros(et.etree_attn_diff_workspace_size(c.batch, 4, 2), dtype=torch.uint8, device="cuda")
    c.call()
    assert et.etree_device_status(c.ws) == (0, 0)
    assert torch.equal(c.out[:c.nt], out) and torch.equal(c.lse[:c.nt], lse)
    assert (c.out[c.nt:] == 7.0).all() and (c.lse[c.nt:] == 7.0).all()
