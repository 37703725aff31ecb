"""Which bits of a token reach the products: with weights that pick single entries
out (one nonzero weight a column), an output is an entry itself, and equal to it
bit for bit where the entry is kept whole."""
import pytest
import torch

from nvfp4_post_weight_b200 import binding as B
from test_gpu_gemv import BF16, DEV, F32, fp4

pytestmark = pytest.mark.gpu
ONE = 56                                       # E4M3 code of 1


def pick(columns, d_in, code=2, sg=1.0):
    """Weights of 1 (E2M1 code 2) at (o, columns[o])."""
    d_out = len(columns)
    codes = torch.zeros((d_out, d_in), dtype=torch.uint8, device=DEV)
    codes[torch.arange(d_out, device=DEV), columns] = code
    packed = (codes[:, 0::2] | codes[:, 1::2] << 4).contiguous()
    return (packed, torch.full((d_out, d_in // 16), ONE, dtype=torch.uint8, device=DEV),
            torch.full((1,), sg, device=DEV))


def bf16_tokens(n, d, octaves, seed):
    """Entries of random bits whose block's largest is at most `octaves` octaves
    above the least; every block has both."""
    g = torch.Generator().manual_seed(seed)
    x = torch.rand((n, d), generator=g) + 1
    down = torch.randint(0, octaves + 1, (n, d), generator=g).float()
    down[:, 0::16], down[:, 9::16] = 0, octaves
    sign = torch.randint(0, 2, (n, d), generator=g) * 2 - 1
    # (below 2 before and after the rounding: the largest lies in [1, 2))
    return (x.clamp(max=1.99) * sign * torch.exp2(-down)).to(BF16).to(DEV)


# one and two panels a stage, tiles of several sizes, K in two parts (from 10240 on)
FP4_SIZES = [(256, 150000), (512, 40000), (1280, 20000), (10240, 8001), (12288, 5201)]


@pytest.mark.parametrize("d_in,d_out", FP4_SIZES)
@pytest.mark.parametrize("n", [3, 17, 40])
def test_fp4_entries_within_20_octaves_are_whole(d_in, d_out, n):
    assert fp4(n, d_out, d_in)
    x = bf16_tokens(n, d_in, 20, n)
    columns = torch.arange(d_out, device=DEV) * 7919 % d_in
    y = torch.empty((n, d_out), device=DEV)
    B.nvfp4_gemv(x, *pick(columns, d_in), y)
    assert torch.equal(y, x.float()[:, columns])


@pytest.mark.parametrize("d_in,d_out", [(512, 20000), (2048, 9505), (8192, 5001)])
@pytest.mark.parametrize("n", [3, 25])
def test_fp4_pair_keeps_entries_whole(d_in, d_out, n):
    """Of the pair, with a gate of 128 everywhere: silu(128) is 128 in fp32."""
    assert fp4(n, d_out, d_in, 0, True)
    x = bf16_tokens(n, d_in, 20, n)
    x[:, 0] = 1.0
    columns = torch.arange(d_out, device=DEV) * 7919 % d_in
    gate = pick(torch.zeros_like(columns), d_in, sg=128.0)
    y = torch.empty((n, d_out), device=DEV)
    B.nvfp4_gemv_swiglu(x, gate, pick(columns, d_in), y)
    assert torch.equal(y, 128 * x.float()[:, columns])


@pytest.mark.parametrize("d_in,d_out", [(512, 13007), (8192, 1000)])
def test_fp4_experts_keep_entries_whole(d_in, d_out):
    counts = [3, 0, 17, 1, 33, 8]
    E, n = len(counts), sum(counts)
    assert fp4(n, d_out, d_in, E)
    x = bf16_tokens(n, d_in, 20, 5)
    columns = torch.arange(d_out, device=DEV) * 7919 % d_in
    codes, scales, _ = pick(columns, d_in)
    offsets = torch.tensor([0, *torch.tensor(counts).cumsum(0)], dtype=torch.int32, device=DEV)
    sg = 2.0 ** torch.arange(E, dtype=F32, device=DEV)
    y = torch.empty((n, d_out), device=DEV)
    B.nvfp4_gemv_experts(x, offsets, codes.repeat(E, 1, 1), scales.repeat(E, 1, 1), sg, y)
    scale = torch.repeat_interleave(sg, torch.tensor(counts, device=DEV))
    assert torch.equal(y, scale[:, None] * x.float()[:, columns])


def fp32_tokens(n, d, seed):
    g = torch.Generator().manual_seed(seed)
    bits = torch.randint(0, 1 << 24, (n, d), generator=g).float() / 2 ** 23 - 1
    return (bits * torch.exp2(torch.randint(-30, 30, (n, d), generator=g).float())).to(DEV)


# odd numbers of blocks, rows that are staged in several parts, K in slices
@pytest.mark.parametrize("d_in,d_out", [(16, 40), (272, 300), (1040, 1040), (4112, 4001),
                                        (8192, 130), (2048, 20000)])
@pytest.mark.parametrize("n", [1, 9, 20, 40])
@pytest.mark.parametrize("xt", [F32, BF16])
def test_general_kernel_keeps_every_bit(d_in, d_out, n, xt):
    """fp32 tokens are three bf16 pieces, all of them used; bf16 ones are whole."""
    x = fp32_tokens(n, d_in, n).to(xt)
    if xt == BF16 and fp4(n, d_out, d_in):
        pytest.skip("runs on the FP4 tensor cores")
    columns = torch.arange(d_out, device=DEV) * 7919 % d_in
    w = pick(columns, d_in)
    y = torch.empty((n, d_out), device=DEV)
    B.nvfp4_gemv(x, *w, y)
    assert torch.equal(y, x.float()[:, columns])
    x[:, 0] = 1.0
    if xt == F32 or not fp4(n, d_out, d_in, 0, True):
        B.nvfp4_gemv_swiglu(x, pick(torch.zeros_like(columns), d_in, sg=128.0), w, y)
        assert torch.equal(y, 128 * x.float()[:, columns])


@pytest.mark.parametrize("d_in,d_out", [(272, 300), (4112, 500)])
def test_general_kernel_keeps_every_bit_by_expert(d_in, d_out):
    counts = [3, 0, 17, 1, 33, 8]
    E, n = len(counts), sum(counts)
    x = fp32_tokens(n, d_in, 5)
    columns = torch.arange(d_out, device=DEV) * 7919 % d_in
    codes, scales, _ = pick(columns, d_in)
    offsets = torch.tensor([0, *torch.tensor(counts).cumsum(0)], dtype=torch.int32, device=DEV)
    sg = 2.0 ** torch.arange(E, dtype=F32, device=DEV)
    rows = torch.randperm(n, device=DEV).int()
    y = torch.empty((n, d_out), device=DEV)
    B.nvfp4_gemv_experts(x, offsets, codes.repeat(E, 1, 1), scales.repeat(E, 1, 1), sg, y, rows)
    scale = torch.repeat_interleave(sg, torch.tensor(counts, device=DEV))
    assert torch.equal(y, scale[:, None] * x[rows.long()][:, columns])


def outlier_tokens(n, d, seed):
    """Entries of N(0, 1), of many octaves, with outliers of 2^4 to 2^100 in some
    blocks, and blocks of zeros and of very small entries."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, d), generator=g)
    x = x * torch.exp2(-torch.randint(0, 24, (n, d), generator=g).float())
    for t in range(n):
        x[t, 32:64] = 0
        x[t, 64:80] *= 2.0 ** -60
        for k, e in enumerate((4, 5, 6, 7, 10, 14, 20) if t % 3 else (22, 30, 60, 100)):
            x[t, (97 + 48 * k) % d] = 1.5 * 2.0 ** e
    return x.to(BF16).to(DEV)


def tops(x, group):
    """Exponents of the largest of every `group` entries, far below all for zeros."""
    top = x.float().abs().unflatten(1, (-1, group)).amax(2)
    return torch.where(top > 0, torch.frexp(top)[1].double() - 1, -1000.0)


def kept(got, x, columns, scale=1.0):
    """Entries to 2^-20 of 2^m, m the mean exponent of the largest of every eight that
    are not all zero; whole in blocks whose largest is 2^8 above 2^m, and where they
    are within 2^-20 of the largest.  (A block counts as no more than 17 octaves below
    the token's largest entry: digits reach no further down.)"""
    e = tops(x, 8)
    m = torch.where(e > -1000, e, 0.0).sum(1, keepdim=True) / (e > -1000).sum(1, keepdim=True)
    top = tops(x, 16)
    top = torch.maximum(top, top.amax(1, keepdim=True) - 17).repeat_interleave(16, 1)[:, columns]
    x, got = x.double()[:, columns], got.double() / scale
    assert ((got - x).abs() <= torch.exp2(m - 20)).all()
    whole = (top > m + 8) | (x.abs() >= torch.exp2(top - 20))
    assert (got == x)[whole].all() and whole.any()


@pytest.mark.parametrize("d_in,d_out", FP4_SIZES)
@pytest.mark.parametrize("n", [3, 40])
def test_fp4_entries_beside_outliers(d_in, d_out, n):
    assert fp4(n, d_out, d_in)
    x = outlier_tokens(n, d_in, n)
    columns = torch.arange(d_out, device=DEV) * 7919 % d_in
    y = torch.empty((n, d_out), device=DEV)
    B.nvfp4_gemv(x, *pick(columns, d_in), y)
    kept(y, x, columns)


@pytest.mark.parametrize("d_in,d_out", [(512, 20000), (8192, 5001)])
def test_fp4_pair_beside_outliers(d_in, d_out):
    n = 25
    assert fp4(n, d_out, d_in, 0, True)
    x = outlier_tokens(n, d_in, n)
    x[:, 0] = 1.0
    columns = torch.arange(d_out, device=DEV) * 7919 % d_in
    gate = pick(torch.zeros_like(columns), d_in, sg=128.0)
    y = torch.empty((n, d_out), device=DEV)
    B.nvfp4_gemv_swiglu(x, gate, pick(columns, d_in), y)
    # (1 is within 2^-20 of its block's largest, or in one that is completed: whole)
    kept(y, x, columns, 128.0)


@pytest.mark.parametrize("d_in,d_out", [(512, 13007), (8192, 1000)])
def test_fp4_experts_beside_outliers(d_in, d_out):
    counts = [3, 0, 17, 1, 33, 8]
    E, n = len(counts), sum(counts)
    assert fp4(n, d_out, d_in, E)
    x = outlier_tokens(20, d_in, 9)
    rows = torch.randint(0, 20, (n,), dtype=torch.int32, device=DEV)
    columns = torch.arange(d_out, device=DEV) * 7919 % d_in
    codes, scales, _ = pick(columns, d_in)
    offsets = torch.tensor([0, *torch.tensor(counts).cumsum(0)], dtype=torch.int32, device=DEV)
    y = torch.empty((n, d_out), device=DEV)
    B.nvfp4_gemv_experts(x, offsets, codes.repeat(E, 1, 1), scales.repeat(E, 1, 1),
                         torch.ones(E, device=DEV), y, rows)
    kept(y, x[rows.long()], columns)


def test_fp4_completes_the_same_bits_in_graphs():
    """The record of what is left out lies in the workspace: two calls of other tokens
    in one captured workspace, replayed, beside eager ones."""
    d_in, d_out, n = 512, 40000, 5
    columns = torch.arange(d_out, device=DEV) * 7919 % d_in
    w = pick(columns, d_in)
    xs = [outlier_tokens(n, d_in, s) for s in (1, 2)] + [bf16_tokens(n, d_in, 3, 3)]
    ws = B.workspace(B.nvfp4_gemv_workspace_size(n, d_out, d_in), DEV)
    ys, zs = ([torch.empty((n, d_out), device=DEV) for _ in xs] for _ in range(2))
    for x, y in zip(xs, ys):
        B.nvfp4_gemv(x, *w, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x, z in zip(xs, zs):
            B.nvfp4_gemv(x, *w, z, ws)
    for _ in range(3):
        ws.fill_(255)
        graph.replay()
    torch.cuda.synchronize()
    for y, z in zip(ys, zs):
        assert torch.equal(y, z)


def test_general_kernel_keeps_entries_beside_outliers():
    d_in, d_out, n = 512, 130, 9
    assert not fp4(n, d_out, d_in)
    x = outlier_tokens(n, d_in, n)
    columns = torch.arange(d_out, device=DEV) * 7919 % d_in
    y = torch.empty((n, d_out), device=DEV)
    B.nvfp4_gemv(x, *pick(columns, d_in), y)
    assert torch.equal(y, x.float()[:, columns])
