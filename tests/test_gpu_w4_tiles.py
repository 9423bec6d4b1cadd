"""Products with 4-bit weights in the kernel that keeps them in tensor memory.

Up to 8 tokens, and small products of up to 64, go to a kernel with one launch; most cases beside these
are small enough for it.  Here every case is one of the other kernel's: more than 64 tokens at any size, or
sizes where it takes over.  Only that kernel writes its workspace behind the status header, and each
case asserts that it did.  Definitions and tolerances are those of the other cases.
"""
import pytest
import torch

import draft_tree_verification_masked_b200 as et

from .test_gpu_w4 import Case

pytestmark = pytest.mark.gpu


def used_tensor_memory(c):
    return bool((c.ws[256:] != 0xA5).any())


def run(c, cols=slice(None)):
    c.call()
    c.check(cols)
    assert used_tensor_memory(c)
    return c


def some(N):
    """Every seventh output column, and the last ones."""
    return torch.cat([torch.arange(0, N, 7), torch.arange(max(0, N - 40), N)])


# tokens a tile, row tiles a unit, then a size there
SHAPES = [(16, 2, 9, 38100, 1440), (16, 2, 16, 38401, 1408), (16, 4, 12, 14001, 4096),
          (16, 4, 16, 13795, 4224), (32, 2, 32, 38100, 768), (32, 2, 17, 37889, 896),
          (32, 4, 20, 7100, 4096), (32, 4, 31, 6901, 4224), (64, 2, 64, 9000, 2048),
          (64, 2, 40, 39000, 640), (64, 2, 65, 1001, 2176), (64, 2, 130, 513, 1152)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("nt,ks,M,N,K", SHAPES)
def test_every_tile_shape_and_group(nt, ks, M, N, K, group):
    K = K // group * group
    # the shape that the plan picks: tokens of a tile from M, two row tiles a unit where they fill the SMs
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert nt == (16 if M <= 16 else 32 if M <= 32 else 64)
    assert ks == (2 if nt == 64 or (N + 255) // 256 >= sms else 4)
    run(Case(M, N, K, group, zeros=M % 2 == 0, bias=M % 3 > 0, f32=M % 4 == 0, seed=M + group),
        some(N))


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 288, 384, 512, 544, 1056, 4992])
@pytest.mark.parametrize("M", [65, 130])
def test_depths_around_blocks(K, M):
    run(Case(M, 130, K, 128 if K % 128 == 0 else 32, seed=K, zeros=K % 64 == 0, f32=True))


@pytest.mark.parametrize("N", [1, 2, 31, 127, 128, 129, 255, 256, 257, 500, 1000, 5120])
@pytest.mark.parametrize("M", [65, 96, 129])
def test_row_counts(N, M):
    run(Case(M, N, 640, 64, seed=N, bias=N % 2 == 0, f32=M == 96))


@pytest.mark.parametrize("M", [65, 127, 128, 193, 700])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_token_counts(M, group):
    run(Case(M, 200, 1280, group, seed=M + group, f32=M % 2 == 0))


@pytest.mark.parametrize("M,N,K,group", [(65, 300, 512, 128), (130, 301, 544, 32), (12, 13801, 4096, 64),
                                         (24, 38100, 704, 64)])
def test_strided_rows(M, N, K, group):
    """x inside a wider buffer whose other columns hold NaN, out inside a wider one."""
    run(Case(M, N, K, group, x_pad=24, out_pad=5, seed=1, f32=M == 130), some(N))


@pytest.mark.parametrize("M,N,K", [(65, 100, 128), (13, 13801, 4096), (25, 38100, 704)])
def test_zero_points_outside_four_bits_use_the_low_bits(M, N, K):
    c = Case(M, N, K, 64, seed=2)
    c.z += 0xB0
    run(c, some(N))


@pytest.mark.parametrize("M,N,K,group", [(65, 150, 512, 128), (66, 150, 512, 32), (14, 13801, 4096, 64)])
def test_extreme_scales(M, N, K, group):
    c = Case(M, N, K, group, seed=5, bias=False, f32=True)
    c.s_h[::3] *= 1e30
    c.s_h[1::3] *= 1e-30
    c.s.copy_(c.s_h)
    run(c, some(N))


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("M,N,K", [(65, 300, 256), (130, 129, 96), (10, 13801, 4096), (10, 38100, 1440),
                                   (20, 7100, 4096), (20, 38100, 768), (40, 38100, 384)])
def test_a_row_that_is_not_finite_stays_alone(value, M, N, K):
    """The last token is not finite at the first, a middle and the last k: other tokens keep their bits, and
    every weight that it meets makes its outputs not finite."""
    c = Case(M, N, K, 32, seed=6, f32=True)
    c.call()
    assert used_tensor_memory(c)
    clean = c.out.clone()
    at = [0, K // 2, K - 1]
    c.x[M - 1, at] = value
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(c.out[:M - 1], clean[:M - 1])
    q = torch.stack([c.wq_h & 15, c.wq_h >> 4], 2).reshape(N, K)[:, at]
    groups = [k // 32 for k in at]
    hit = ((q != c.z_h[:, groups]) & (c.s_h[:, groups] != 0)).any(1)
    assert hit.any() and (~torch.isfinite(c.out[M - 1])).cpu()[hit].all()


@pytest.mark.parametrize("M,N,K", [(65, 1000, 5120), (12, 13801, 4096), (20, 7100, 4096), (130, 513, 544)])
def test_results_do_not_depend_on_the_run(M, N, K):
    c = Case(M, N, K, 32, seed=7)
    c.call()
    assert used_tensor_memory(c)
    first = c.out.clone()
    for _ in range(20):
        c.out.fill_(0)
        c.call()
        assert torch.equal(c.out, first)


def test_replays_from_graphs_on_two_streams():
    cs = [Case(65, 700, 1024, 128, seed=8), Case(20, 7100, 4096, 64, seed=9), Case(130, 900, 512, 32, seed=10)]
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
        c.check(some(c.N))
        assert used_tensor_memory(c)


def test_two_calls_in_turn_share_a_workspace():
    """The second call's sizes differ: nothing of the first is taken for its own."""
    a, b = Case(130, 900, 1024, 64, seed=11), Case(65, 1500, 544, 32, seed=12)
    ws = torch.zeros(max(a.ws.numel(), b.ws.numel()), dtype=torch.uint8, device="cuda")
    for c in (a, b, a, b):
        c.out.fill_(0)
        et.etree_w4_linear(c.x, c.wq, c.s, c.z, c.group, c.b, c.out, ws)
        c.check()
    assert et.etree_device_status(ws) == (0, 0)
