"""GPU checks of the embedding lookup (bit for bit: one fp32 product, rounded
once) and of its gradient: per element at most n + 2 roundings of fp32 (n the
number of tokens that name the row) on the sum of magnitudes, against the
64-bit sum; zeros where no token names a row; the same bits every time."""
import pytest
import torch

import bit_block_scaled_quant_amd as nv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def tokens(T, V, seed, kind="zipf"):
    g = torch.Generator(device=DEV).manual_seed(seed)
    u = torch.rand(T, generator=g, device=DEV)
    t = (torch.pow(float(V), u).long() - 1 if kind == "zipf" else (u * V).long()).clamp(0, V - 1)
    bad = torch.rand(T, generator=g, device=DEV) < 0.05
    return torch.where(bad, torch.full_like(t, -1), t).int(), g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (3, 5, 7), (9, 40, 8), (65, 100, 63), (100, 1000, 64), (33, 77, 515),
                                   (1000, 300, 1027), (2049, 5000, 2056), (17, 64, 5120)])
def test_lookup(T, V, D, dtype):
    tok, g = tokens(T, V, T + D)
    tok[-1] = V  # outside above
    table = torch.randn(V, D, generator=g, device=DEV).to(dtype)
    for scale in (1.0, D ** 0.5, -0.3):
        ok = (tok >= 0) & (tok < V)
        want = table[tok.long().clamp(0, V - 1)].float() * torch.tensor(scale, dtype=torch.float32, device=DEV)
        want = torch.where(ok[:, None], want, torch.zeros_like(want)).to(dtype)
        assert torch.equal(nv.embed(tok, table, scale=scale), want)


def check_grad(tok, dout, V, scale):
    D = dout.shape[1]
    got = nv.embed_grad(tok, dout, V, scale=scale)
    ok = (tok >= 0) & (tok < V)
    at, x = tok[ok].long(), dout[ok].double()
    want = torch.zeros(V, D, dtype=torch.float64, device=DEV).index_add_(0, at, x) * float(torch.tensor(scale))
    mag = torch.zeros(V, D, dtype=torch.float64, device=DEV).index_add_(0, at, x.abs()) * abs(scale)
    n = torch.zeros(V, dtype=torch.float64, device=DEV).index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    assert (got[n == 0] == 0).all()
    assert ((got.double() - want).abs() <= (n + 2)[:, None] * 2.0 ** -24 * mag).all()
    assert torch.equal(got, nv.embed_grad(tok, dout, V, scale=scale))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 1000, 64), (5, 3, 7), (64, 64, 64), (257, 30, 63), (1000, 1000, 65),
                                   (4095, 200, 130), (4097, 1000, 256), (8192, 1000, 96), (300, 5000, 1027),
                                   (2000, 100, 2051), (513, 70000, 80), (9001, 33, 260), (8192, 20000, 1032), (16384, 50, 16),
                                   (30000, 3000, 40), (70001, 500, 20)])
@pytest.mark.parametrize("kind", ["zipf", "even"])
def test_gradient(T, V, D, dtype, kind):
    tok, g = tokens(T, V, T + V, kind)
    check_grad(tok, torch.randn(T, D, generator=g, device=DEV).to(dtype), V, 1.7)


@pytest.mark.parametrize("D", [64, 1027])
def test_gradient_of_one_row(D):  # every token names it
    dout = torch.randn(6000, D, device=DEV).bfloat16()
    for v in (0, 63, 64, 199):
        check_grad(torch.full((6000,), v, dtype=torch.int32, device=DEV), dout, 200, 0.5)


def test_gradient_of_many_rows_in_one_workgroup():  # every row of a range named, over and over
    tok = (torch.arange(12000, device=DEV) * 7 % 64 + 64 * 3).int()
    check_grad(tok, torch.randn(12000, 72, device=DEV), 200000, 1.0)


@pytest.mark.parametrize("times", [7, 8, 9, 10])
@pytest.mark.parametrize("T", [8191, 8192, 8193])
def test_gradient_of_rows_named_equally_often(T, times):
    """Rows on either side of the border between short and long ones, as many long
    ones as fit, the last row of the table among them."""
    V = (T + times - 1) // times
    g = torch.Generator(device=DEV).manual_seed(T)
    tok = (torch.arange(T, device=DEV) // times)[torch.randperm(T, generator=g, device=DEV)].int()
    check_grad(tok, torch.randn(T, 36, generator=g, device=DEV).bfloat16(), V, 1.0)


def test_gradient_ignores_tokens_outside():
    tok = torch.tensor([-1, 50, 2 ** 31 - 1, -2 ** 31, 3, 51, 49], dtype=torch.int32, device=DEV)
    check_grad(tok, torch.randn(7, 33, device=DEV), 50, 2.0)


def test_no_tokens():
    tok = torch.empty(0, dtype=torch.int32, device=DEV)
    assert nv.embed(tok, torch.randn(4, 6, device=DEV)).shape == (0, 6)
    grad = torch.full((100, 6), 3.0, device=DEV)
    nv.nvfp4_embed_grad(tok, torch.empty(0, 6, device=DEV), 1.0, grad, torch.empty(0, dtype=torch.uint8, device=DEV))
    assert not grad.any()


def test_gradient_against_differences():
    """A step in one table entry moves sum(out * dout) by grad times the step
    (the lookup is linear, so the difference is exact up to its roundings)."""
    tok, g = tokens(50, 9, 3)
    table, dout = torch.randn(9, 5, device=DEV), torch.randn(50, 5, device=DEV)
    grad = nv.embed_grad(tok, dout, 9, scale=2.5)
    base = (nv.embed(tok, table, scale=2.5).double() * dout.double()).sum()
    for v, d in ((0, 0), (1, 4), (3, 2), (8, 1)):
        moved = table.clone()
        moved[v, d] += 1.0
        diff = (nv.embed(tok, moved, scale=2.5).double() * dout.double()).sum() - base
        assert abs(diff.item() - grad[v, d].item()) < 1e-4


@pytest.mark.parametrize("T,V,D", [(100, 50, 5), (100, 50, 67), (1, 1, 1030)])
def test_nothing_outside_the_outputs_is_written(T, V, D):
    tok, g = tokens(T, V, 1)
    space = torch.empty(nv.nvfp4_embed_grad_workspace(T), dtype=torch.uint8, device=DEV)
    for rows, call in ((T, lambda o: nv.nvfp4_embed(tok, torch.ones(V, D, device=DEV), 1.0, o)),
                       (V, lambda o: nv.nvfp4_embed_grad(tok, torch.ones(T, D, device=DEV), 1.0, o, space))):
        buf = torch.full((rows * D + 256,), 7.25, device=DEV)
        call(buf[128:128 + rows * D].view(rows, D))
        assert (buf[:128] == 7.25).all() and (buf[128 + rows * D:] == 7.25).all()


def test_large_table():
    """Element offsets past 2^31 (the table's gradient alone is 8.6 GB)."""
    V, D = 2 ** 21 + 3, 1024
    tok = torch.tensor([0, V - 1, 2 ** 20, 2 ** 21, -1, V - 1], dtype=torch.int32, device=DEV)
    dout = torch.randn(6, D, device=DEV)
    grad = nv.embed_grad(tok, dout, V)
    assert torch.equal(grad[2 ** 20], dout[2]) and torch.equal(grad[2 ** 21], dout[3])
    assert torch.equal(grad[V - 1], dout[1] + dout[5])
    assert grad.view(-1).count_nonzero().item() == grad[[0, 2 ** 20, 2 ** 21, V - 1]].count_nonzero().item()
    out = nv.embed(tok, grad)
    assert torch.equal(out[1], grad[V - 1]) and torch.equal(out[3], grad[2 ** 21])


@pytest.mark.parametrize("T", [700, 9000])
def test_workspace_contents_do_not_matter(T):
    V, D = 300, 20
    tok, g = tokens(T, V, 2)
    dout = torch.randn(T, D, device=DEV)
    want, got = nv.embed_grad(tok, dout, V), torch.empty(V, D, device=DEV)
    size = nv.nvfp4_embed_grad_workspace(T)
    for fill in (0, 0xFF):
        nv.nvfp4_embed_grad(tok, dout, 1.0, got, torch.full((size,), fill, dtype=torch.uint8, device=DEV))
        assert torch.equal(got, want)
    space = torch.zeros(size // 4, dtype=torch.int32, device=DEV)  # indexes of another call
    space.copy_(torch.arange(size // 4, device=DEV) % T)
    nv.nvfp4_embed_grad(tok, dout, 1.0, got, space.view(torch.uint8))
    assert torch.equal(got, want)
