"""Products with 4-bit weights on the GPU against their fp64 definition.

Tolerances.  q - z and its product with a bf16 x are exact in fp32.  A group's sum is made of at
most 128 additions by the tensor core, each off by at most 2^-23 of the magnitudes added so far;
the scaled sums meet in fp32 with one rounding a group (2^-24), and the partial sums of a row tile
and the bias in fewer than 160 more.  So with mass = sum |x (q - z) s| + |b|,
  |out - exact| <= (128 * 2^-23 + (K / group + 160) * 2^-24) mass + r |exact|,
where r is the output's rounding, 2^-8 for bf16 and 2^-24 for fp32.
"""
import numpy as np
import pytest
import torch

import draft_tree_verification_masked_b200 as et
from oracle import serving as S

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, M, N, K, group, zeros=True, bias=True, f32=False, x_pad=0, out_pad=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.M, self.N, self.K, self.group, self.f32 = M, N, K, group, f32
        bf = torch.bfloat16
        self.x_h = torch.randn(M, K + x_pad, generator=g).to(bf)[:, :K]
        self.wq_h = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=g)
        self.s_h = (0.01 * torch.randn(N, K // group, generator=g)).to(bf)
        self.z_h = torch.randint(0, 16, (N, K // group), dtype=torch.uint8,
                                 generator=g) if zeros else None
        self.b_h = torch.randn(N, generator=g).to(bf) if bias else None
        self.x = torch.full((M, K + x_pad), float("nan"), dtype=bf, device="cuda")[:, :K]
        self.x.copy_(self.x_h)
        self.wq, self.s = self.wq_h.cuda(), self.s_h.cuda()
        self.z = None if self.z_h is None else self.z_h.cuda()
        self.b = None if self.b_h is None else self.b_h.cuda()
        dt = torch.float32 if f32 else bf
        self.out_g = torch.full((M + 2, N + out_pad), 7.0, dtype=dt, device="cuda")
        self.out = self.out_g[1:-1, :N]
        size = et.etree_w4_workspace_size(M, N, K)
        # a used workspace: only its header is zero
        self.ws_g = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        self.ws = self.ws_g[256:-256]
        self.ws[:256] = 0

    def call(self, stream=None):
        et.etree_w4_linear(self.x, self.wq, self.s, self.z, self.group, self.b, self.out, self.ws,
                           stream)

    def exact(self, cols=slice(None)):
        x = self.x_h.double().numpy()
        q = self.wq_h[cols].numpy()
        s, z = self.s_h[cols].double().numpy(), None if self.z_h is None else self.z_h[cols].numpy()
        b = None if self.b_h is None else self.b_h[cols].double().numpy()
        w = S.w4_weights(q, s, z, self.group)
        y = S.w4_linear(x, q, s, z, self.group, b)
        mass = np.abs(x) @ np.abs(w).T + (0 if b is None else np.abs(b))
        return y, mass

    def check(self, cols=slice(None)):
        torch.cuda.synchronize()
        assert et.etree_device_status(self.ws) == (0, 0)
        assert (self.ws_g[:256] == 0xA5).all() and (self.ws_g[-256:] == 0xA5).all()
        assert (self.out_g[0] == 7.0).all() and (self.out_g[-1] == 7.0).all()
        assert (self.out_g[:, self.N:] == 7.0).all()
        y, mass = self.exact(cols)
        tol = (128 * 2.0 ** -23 + (self.K / self.group + 160) * 2.0 ** -24) * mass
        tol += (2.0 ** -24 if self.f32 else 2.0 ** -8) * np.abs(y) + 1e-38
        got = self.out[:, cols].double().cpu().numpy()
        bad = ~(np.abs(got - y) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:5], bad.mean())
        return self

    def run(self):
        self.call()
        return self.check()


@pytest.mark.parametrize("M", [1, 2, 5, 16, 17, 32, 33, 64, 65, 130])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_tokens_and_groups(M, group):
    Case(M, 200, 1280, group, seed=M + group, f32=M % 2 == 0).run()


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 288, 384, 512, 544, 1056, 4992])
@pytest.mark.parametrize("M", [1, 20, 40])
def test_depths_around_blocks(K, M):
    group = 128 if K % 128 == 0 else 32
    Case(M, 130, K, group, seed=K, zeros=K % 64 == 0, f32=True).run()


@pytest.mark.parametrize("N", [1, 2, 31, 127, 128, 129, 500, 1000, 5120])
@pytest.mark.parametrize("M", [1, 7, 48])
def test_row_counts(N, M):
    Case(M, N, 640, 64, seed=N, bias=N % 2 == 0).run()


@pytest.mark.parametrize("M,group", [(1, 32), (16, 64), (24, 32), (64, 32), (64, 64), (64, 128),
                                     (70, 128)])
@pytest.mark.parametrize("f32", [False, True])
def test_many_rows(M, group, f32):
    """Enough rows that a unit is four row tiles."""
    Case(M, 38100, 384, group, seed=M, f32=f32).run()


@pytest.mark.parametrize("M,N,K,group", [
    (12, 14001, 4096, 32), (16, 13800, 4096, 128), (9, 38100, 1408, 128), (16, 38100, 1408, 64),
    (20, 7100, 4096, 64), (32, 7000, 4096, 128), (31, 6900, 4160, 32), (17, 38100, 704, 64),
    (32, 38100, 768, 32), (64, 9000, 2048, 128), (40, 39000, 704, 32)])
def test_large_products_of_few_tokens(M, N, K, group):
    """Where the kernel without tensor memory gives way to the other, at each of its shapes; every
    seventh output column and the last ones are compared."""
    c = Case(M, N, K, group, seed=M, zeros=M % 2 == 0, f32=M % 3 == 0)
    c.call()
    c.check(torch.cat([torch.arange(0, N, 7), torch.arange(N - 40, N)]))


def test_many_token_chunks():
    Case(200, 13000, 128, 128, seed=3).run()


def test_strided_rows():
    """x inside a wider buffer, out inside a wider one: the other columns stay as they were."""
    Case(9, 300, 512, 128, x_pad=24, out_pad=5, seed=1).run()
    Case(40, 300, 512, 32, x_pad=8, out_pad=3, seed=1, f32=True).run()


def test_zero_points_outside_four_bits_use_the_low_bits():
    c = Case(3, 100, 128, 64, seed=2)
    c.z += 0xB0
    c.run()


def test_extreme_scales_and_values():
    c = Case(4, 150, 512, 128, seed=5, bias=False, f32=True)
    c.s_h[::3] *= 1e30
    c.s_h[1::3] *= 1e-30
    c.s.copy_(c.s_h)
    c.run()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_row_that_is_not_finite_stays_alone(value):
    for M, N in ((8, 300), (40, 38100)):
        c = Case(M, N, 256, 64, seed=6)
        c.call()
        clean = c.out.clone()
        c.x[3, 17] = value
        c.call()
        torch.cuda.synchronize()
        keep = [i for i in range(M) if i != 3]
        assert torch.equal(c.out[keep], clean[keep])
        moved = ~torch.isfinite(c.out[3])
        q = torch.stack([c.wq_h & 15, c.wq_h >> 4], 2).reshape(N, 256)[:, 17]
        hit = (q != c.z_h[:, 0]) & (c.s_h[:, 0] != 0)
        assert moved.cpu()[hit].all()


def test_results_do_not_depend_on_the_run():
    """Many CTAs a tile, replayed: bit for bit the same."""
    for c in (Case(16, 1000, 5120, 64, seed=7), Case(64, 39000, 1024, 128, seed=7)):
        c.call()
        first = c.out.clone()
        for _ in range(5):
            c.out.fill_(0)
            c.call()
            assert torch.equal(c.out, first)


def test_no_tokens_and_refusals():
    c = Case(4, 100, 256, 64)
    out = torch.empty(0, 100, dtype=torch.bfloat16, device="cuda")
    assert et.etree_w4_linear(c.x[:0], c.wq, c.s, c.z, 64, c.b, out, c.ws) == 0
    with pytest.raises(TypeError):
        et.etree_w4_linear(c.x.float(), c.wq, c.s, c.z, 64, c.b, c.out, c.ws)
    with pytest.raises(TypeError):
        et.etree_w4_linear(c.x, c.wq, c.s, c.z, 64, c.b, c.out.half(), c.ws)
    with pytest.raises(ValueError):
        et.etree_w4_linear(c.x, c.wq, c.s, c.z, 32, c.b, c.out, c.ws)
    with pytest.raises(ValueError):
        et.etree_w4_linear(c.x, c.wq[:, :-1], c.s, c.z, 64, c.b, c.out, c.ws)
    with pytest.raises(ValueError):
        et.etree_w4_linear(c.x, c.wq, c.s, c.z, 64, c.b[:-1], c.out, c.ws)
    with pytest.raises(ValueError):
        et.etree_w4_linear(c.x, c.wq, c.s.cpu(), c.z, 64, c.b, c.out, c.ws)
    with pytest.raises(et.EtreeError):
        et.etree_w4_linear(c.x, c.wq, c.s, c.z, 64, c.b, c.out, c.ws[:256])
    with pytest.raises(et.EtreeError):       # rows of x that start off a 16-byte boundary
        x = torch.zeros(4, 260, dtype=torch.bfloat16, device="cuda")[:, 2:258]
        et.etree_w4_linear(x, c.wq, c.s, c.z, 64, c.b, c.out, c.ws)


def test_replays_from_graphs_on_two_streams():
    cs = [Case(5, 700, 1024, 128, seed=8), Case(33, 900, 512, 64, seed=9)]
    graphs, streams = [], [torch.cuda.Stream() for _ in cs]
    for c, s in zip(cs, streams):
        c.call()
        g = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            c.call()
        graphs.append(g)
    for c in cs:
        c.x_h.mul_(-1)
        c.x.mul_(-1)
        c.out.fill_(0)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    for c in cs:
        c.check()
