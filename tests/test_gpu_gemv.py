"""Products of a few tokens with solved NVFP4 weights (nvfp4_gemv, its gated
pair and both by expert) against fp64 products with the dequantised weights.

Tolerances: the products x * e2m1 * e4m3 are exact, so what is left are the
roundings of the fp32 sums.  Along any path from a product to the result there
are at most K / 32 + 160 of them (a lane's share of the row, the steps inside
one 128-column tile, the joins), each at most 2^-23 of the sum of absolute
values S (twice the half step, for units that truncate); then one rounding of
the output, half a step of its type relative to it.
"""
import numpy as np
import pytest
import torch

import oracle as O
from nvfp4_post_weight_b200 import binding as B
from nvfp4_post_weight_b200 import synth
from nvfp4_post_weight_b200.decoder import DecoderLayerSolver
from nvfp4_post_weight_b200.layer import LayerSolver

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def weights(shape, seed, lo=60, hi=127):
    g = torch.Generator().manual_seed(seed)
    *lead, d_out, d_in = shape
    codes = torch.randint(0, 256, (*lead, d_out, d_in // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(lo, hi, (*lead, d_out, d_in // 16), generator=g, dtype=torch.uint8)
    sg = torch.rand(lead[0] if lead else 1, generator=g) * 1e-3 + 1e-3
    return codes.to(DEV), scales.to(DEV), sg.to(DEV)


def dequantised(codes, scales, sg):
    """fp64 weights of one matrix (device)."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    c = codes.long()
    nib = torch.stack((c & 15, c >> 4), -1).reshape(c.shape[0], -1)
    e4m3 = [(8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) if c > 7 else c * 2.0 ** -9 for c in range(128)]
    block = torch.tensor(e4m3, dtype=torch.float64, device=DEV)[(scales & 127).long()]
    mag = grid[nib & 7]
    return torch.where(nib > 7, -mag, mag) * block.repeat_interleave(16, 1) * sg.double()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def sums(x, w):
    """(product, tolerance of its fp32 sum) in fp64."""
    x, q = x.double(), dequantised(*w)
    K = q.shape[1]
    return x @ q.T, (K / 32 + 160) * 2.0 ** -23 * (x.abs() @ q.abs().T)


def gated(x, gate, up):
    """(silu(g) u, tolerance): |silu'| <= 1.1, and eight roundings of expf, the
    sum, the division and the product."""
    (g, dg), (u, du) = sums(x, gate), sums(x, up)
    s = g * torch.sigmoid(g)
    return s * u, 1.1 * u.abs() * dg + s.abs() * du + 1.1 * dg * du + \
        8 * 2.0 ** -23 * (s * u).abs() + 1e-36


def close(y, ref, tol):
    tol = tol + half_step(y.dtype) * (ref.abs() + tol) + 1e-38
    bad = ~((y.double() - ref).abs() <= tol)
    assert not bad.any(), ((y.double() - ref).abs() / tol).max().item()


def acts(n, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, d), generator=g) * torch.exp(torch.randn(d, generator=g))
    return x.to(dtype).to(DEV)


SHAPES = [(1, 1, 16), (1, 16, 128), (3, 17, 144), (8, 33, 512), (9, 100, 1040), (5, 7, 4112),
          (16, 64, 256), (17, 31, 272), (40, 130, 656), (1, 300, 8192), (2, 48, 28672),
          (70, 257, 2064), (129, 24, 96)]


@pytest.mark.parametrize("n_tok,d_out,d_in", SHAPES)
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_gemv(n_tok, d_out, d_in, xt, yt):
    w, x = weights((d_out, d_in), d_out + d_in), acts(n_tok, d_in, xt, n_tok)
    y = torch.full((n_tok, d_out), 7.0, dtype=yt, device=DEV)
    B.nvfp4_gemv(x, *w, y)
    close(y, *sums(x, w))


@pytest.mark.parametrize("n_tok,d_out,d_in", SHAPES)
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (F32, F32)])
def test_gemv_swiglu(n_tok, d_out, d_in, xt, yt):
    gate, up = weights((d_out, d_in), 1 + d_in), weights((d_out, d_in), 2 + d_in)
    x = acts(n_tok, d_in, xt, n_tok) * 0.1
    y = torch.full((n_tok, d_out), 7.0, dtype=yt, device=DEV)
    B.nvfp4_gemv_swiglu(x, gate, up, y)
    close(y, *gated(x, gate, up))


def test_every_code_and_scale():
    """Each element code under each scale code (subnormal ones, 0 and the
    largest among them), one nonzero token entry at a time: exact in fp32."""
    d_in, codes = 16, np.arange(16)
    nib = np.stack([np.roll(codes, r) for r in range(16)])            # 16 x 16
    rows = np.repeat(nib, 128, axis=0)
    packed = (rows[:, 0::2] | (rows[:, 1::2] << 4)).astype(np.uint8)
    scales = np.tile(np.arange(128), 16).astype(np.uint8)[:, None]
    w = (torch.from_numpy(packed).to(DEV), torch.from_numpy(scales).to(DEV),
         torch.ones(1, device=DEV))
    for xt in (BF16, F32):
        x = torch.eye(16, dtype=xt, device=DEV)
        y = torch.empty((16, 2048), dtype=F32, device=DEV)
        B.nvfp4_gemv(x, *w, y)
        assert torch.equal(y.double(), dequantised(*w).T)


def test_fp32_tokens_keep_all_their_bits():
    w = weights((50, 256), 3)
    x = torch.zeros((4, 256), device=DEV)
    x[0, 5], x[1, 17], x[2, 100], x[3, 255] = 1 + 2.0 ** -23, 16777215.0, -3.1415927, 1e-30
    y = torch.empty((4, 50), device=DEV)
    B.nvfp4_gemv(x, *w, y)
    ref = x.double() @ dequantised(*w).T
    # three pieces joined (at most 2^-23 each) and two products
    assert ((y.double() - ref).abs() <= 8 * 2.0 ** -24 * ref.abs()).all()


@pytest.mark.parametrize("xt", [BF16, F32])
def test_extreme_tokens_and_scales(xt):
    """Large and tiny tokens, and global scales near both ends of fp32."""
    for mag, sg in ((1e30, 1e-3), (1e-30, 1e3), (1e3, 1e-36), (1e-3, 1e34)):
        w = weights((40, 528), 11)
        w[2].fill_(sg)
        x = (acts(3, 528, F32, 5) * mag).to(xt)
        y = torch.empty((3, 40), device=DEV)
        B.nvfp4_gemv(x, *w, y)
        ref, tol = sums(x, w)
        assert ((y.double() - ref).abs() <= tol + 2.0 ** -23 * ref.abs() + 2.0 ** -148).all()


@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("n_tok", [3, 20])
def test_nonfinite_tokens_stay_in_their_row(xt, n_tok):
    w, x = weights((70, 272), 21), acts(n_tok, 272, xt, 22)
    x[1, 3], x[2, 200], x[2, 9] = float("nan"), float("inf"), 1.0
    y = torch.empty((n_tok, 70), dtype=F32, device=DEV)
    B.nvfp4_gemv(x, *w, y)
    ref = (x.double()[:, None, :] * dequantised(*w)[None]).sum(-1)
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    inf = torch.isinf(ref)
    assert inf.any() and torch.equal(y[inf].double(), ref[inf])
    keep = [i for i in range(n_tok) if i not in (1, 2)]
    close(y[keep], *sums(x[keep], w))


def test_zero_blocks_and_empty_sizes():
    codes, scales, sg = weights((20, 64), 4)
    scales[3], codes[3] = 0, 0
    x = acts(2, 64, BF16, 1)
    y = torch.full((2, 20), 5.0, device=DEV)
    B.nvfp4_gemv(x, codes, scales, sg, y)
    assert (y[:, 3] == 0).all()
    # no tokens, no outputs, no inputs (an empty sum: zeros, for the pair too)
    B.nvfp4_gemv(x[:0], codes, scales, sg, y[:0])
    B.nvfp4_gemv(x, codes[:0], scales[:0], sg, y[:, :0].contiguous())
    e = (codes[:, :0].contiguous(), scales[:, :0].contiguous(), sg)
    y.fill_(5.0)
    B.nvfp4_gemv(x[:, :0].contiguous(), *e, y)
    assert (y == 0).all()
    y.fill_(5.0)
    B.nvfp4_gemv_swiglu(x[:, :0].contiguous(), e, e, y)
    assert (y == 0).all()


@pytest.mark.parametrize("d_in", [64, 80, 1024, 1040])
def test_unaligned_bases(d_in):
    """Codes 8 bytes off a 16-byte boundary, scales at an odd byte, row slices."""
    w = weights((40, d_in), 8)
    x = acts(3, d_in, BF16, 2)
    ref = sums(x, w)
    codes = torch.empty(w[0].numel() + 8, dtype=torch.uint8, device=DEV)[8:].view(w[0].shape)
    scales = torch.empty(w[1].numel() + 1, dtype=torch.uint8, device=DEV)[1:].view(w[1].shape)
    codes.copy_(w[0])
    scales.copy_(w[1])
    buf = torch.empty(3 * 40 + 1, dtype=BF16, device=DEV)
    y = buf[1:].view(3, 40)
    B.nvfp4_gemv(x, codes, scales, w[2], y)
    close(y, *ref)
    y = torch.empty((3, 21), device=DEV)
    B.nvfp4_gemv(x, codes[19:], scales[19:], w[2], y)
    close(y, ref[0][:, 19:], ref[1][:, 19:])


def test_the_same_call_twice_gives_the_same_bits():
    w, x = weights((300, 2064), 31), acts(6, 2064, BF16, 3)
    ys = [torch.empty((6, 300), device=DEV) for _ in range(2)]
    for y in ys:
        B.nvfp4_gemv(x, *w, y)
    assert torch.equal(*ys)


# ---- by expert ---------------------------------------------------------------
def by_expert(fn, offsets, *ws):
    """fn(row range, matrices of expert e) for every expert with rows."""
    ends = offsets.tolist()
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if b > a:
            fn(slice(a, b), *[tuple((w[0][e], w[1][e], w[2][e])) for w in ws])


COUNTS = [[1], [0, 3, 0, 0, 1, 0], [8, 0, 9, 1, 17, 0, 64], [0, 0, 0], [150, 1]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("d_out,d_in", [(40, 272), (136, 1024)])
@pytest.mark.parametrize("xt,yt", [(BF16, F32), (F32, F32), (BF16, BF16)])
def test_gemv_experts(counts, d_out, d_in, xt, yt):
    E, n = len(counts), sum(counts)
    extra = 5   # rows behind the last expert's stay as they were
    w = weights((E, d_out, d_in), 5 + E)
    x = acts(n + extra, d_in, xt, 9)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    y = torch.full((n + extra, d_out), 7.0, dtype=yt, device=DEV)
    B.nvfp4_gemv_experts(x, offsets, *w, y)
    by_expert(lambda r, m: close(y[r], *sums(x[r], m)), offsets, w)
    assert (y[n:] == 7).all()


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("xt", [BF16, F32])
def test_gemv_swiglu_experts_with_rows(counts, xt):
    E, n, d_out, d_in = len(counts), sum(counts), 72, 400
    gate, up = weights((E, d_out, d_in), 50 + E), weights((E, d_out, d_in), 60 + E)
    x = acts(11, d_in, xt, 9) * 0.1
    rows = torch.randint(0, 11, (n + 3,), dtype=torch.int32, device=DEV)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    y = torch.full((n + 3, d_out), 7.0, dtype=xt, device=DEV)
    B.nvfp4_gemv_swiglu_experts(x, offsets, gate, up, y, rows)
    xr = x[rows.long()]
    by_expert(lambda r, g, u: close(y[r], *gated(xr[r], g, u)), offsets, gate, up)
    assert (y[n:] == 7).all()


def test_bad_offsets_and_rows_are_cut():
    """Offsets beyond the rows are cut to them; a row index outside X reads as
    zeros."""
    w, x = weights((2, 24, 64), 1), acts(4, 64, BF16, 1)
    offsets = torch.tensor([-3, 2, 9], dtype=torch.int32, device=DEV)
    rows = torch.tensor([0, -1, 4, 3, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    y = torch.full((5, 24), 7.0, device=DEV)
    B.nvfp4_gemv_experts(x, offsets, *w, y, rows)
    for r, (e, src) in enumerate([(0, 0), (0, None), (1, None), (1, 3), (1, None)]):
        if src is None:
            assert (y[r] == 0).all()
        else:
            close(y[r:r + 1], *sums(x[src:src + 1], (w[0][e], w[1][e], w[2][e])))


def test_descending_offsets_give_no_rows():
    w, x = weights((2, 24, 64), 1), acts(4, 64, BF16, 1)
    offsets = torch.tensor([3, 1, 2], dtype=torch.int32, device=DEV)
    y = torch.full((4, 24), 7.0, device=DEV)
    B.nvfp4_gemv_experts(x, offsets, *w, y)
    assert (y[[0, 2, 3]] == 7).all()
    close(y[1:2], *sums(x[1:2], (w[0][1], w[1][1], w[2][1])))


def test_offsets_past_32_bits():
    """The last of 1024 experts whose codes lie beyond 2^31 bytes."""
    E, d_out, d_in = 1024, 1100, 4096
    codes = torch.zeros((E, d_out, d_in // 2), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((E, d_out, d_in // 16), dtype=torch.uint8, device=DEV)
    sg = torch.ones(E, device=DEV)
    c, s, g = weights((d_out, d_in), 77)
    codes[-1], scales[-1], sg[-1] = c, s, g[0]
    x = acts(2, d_in, BF16, 4)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:-1], offsets[-1] = 1, 2
    y = torch.full((2, d_out), 7.0, device=DEV)
    B.nvfp4_gemv_experts(x, offsets, codes, scales, sg, y)
    assert (y[0] == 0).all()
    close(y[1:], *sums(x[1:], (c, s, g)))


# ---- streams, graphs and the solvers -------------------------------------------
def test_own_stream_and_graph_replay():
    w, gate, up = weights((200, 512), 1), weights((200, 512), 2), weights((200, 512), 3)
    x, y, z = acts(4, 512, BF16, 1), torch.empty((4, 200), device=DEV), \
        torch.empty((4, 200), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.nvfp4_gemv(x, *w, y, stream=side)
    side.synchronize()
    close(y, *sums(x, w))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.nvfp4_gemv(x, *w, y)
        B.nvfp4_gemv_swiglu(x, gate, up, z)
    for seed in (7, 8):
        x.copy_(acts(4, 512, BF16, seed) * 0.1)
        graph.replay()
        torch.cuda.synchronize()
        close(y, *sums(x, w))
        close(z, *gated(x, gate, up))


def test_a_solved_layer_answers():
    W, X = synth.small_outlier(d_out=64, d_in=256, n_tok=512, seed=0)
    s = LayerSolver(64, 256, DEV, out_dtype=F32)
    s.step(W.to(DEV), X.to(DEV))
    x = X[:5].to(DEV).to(BF16)
    y = s.linear(x, torch.empty((5, 64), device=DEV))
    ref = O.solve_layer(W.double().numpy(), X.double().numpy())
    q = dequantised(s.codes, s.scales, s.s_g)
    assert np.float32(s.s_g.item()) == ref["s_g"]
    assert torch.equal(q.float(), s.Q)
    close(y, *sums(x, (s.codes, s.scales, s.s_g)))
    assert s.linear(x).dtype == BF16


def test_a_solved_decoder_layer_answers():
    groups = (("x", {"gate": (96, 64), "up": (96, 64)}), ("h", {"down": (64, 96)}))
    s = DecoderLayerSolver(groups, DEV)
    g = torch.Generator().manual_seed(1)
    Ws = {n: (torch.randn(shape, generator=g) * 0.1).to(BF16).to(DEV)
          for n, shape in s.shapes.items()}
    s.step(Ws, {"x": acts(300, 64, BF16, 1), "h": acts(300, 96, BF16, 2)})
    x = acts(3, 64, BF16, 3)
    h = s.gated("gate", "up", x)
    close(h, *gated(x, s.weight("gate"), s.weight("up")))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = s.linear("down", h, stream=side)
    side.synchronize()
    close(y, *sums(h, s.weight("down")))


# ---- the block-scaled FP4 tensor-core path ---------------------------------------
def fp4(n_rows, d_out, d_in, n_experts=0, pair=False):
    """Whether bf16 tokens of these sizes run there (fp32 ones do not)."""
    return B.nvfp4_gemv_workspace_size(n_rows, d_out, d_in, n_experts, pair) > 0


def sums_fp4(x, w):
    """sums() with what the digits leave out of a token: 2^-22 of the largest of
    each block of 16 entries, or 2^-39 of the token's largest."""
    x64 = x.double()
    top = x64.abs().unflatten(1, (-1, 16)).amax(2)
    left = torch.maximum(top * 2.0 ** -22, x64.abs().amax(1, keepdim=True) * 2.0 ** -39)
    q = dequantised(*w)
    y, tol = sums(x, w)
    return y, tol + left.repeat_interleave(16, 1) @ q.abs().T


def gated_fp4(x, gate, up):
    (g, dg), (u, du) = sums_fp4(x, gate), sums_fp4(x, up)
    s = g * torch.sigmoid(g)
    return s * u, 1.1 * u.abs() * dg + s.abs() * du + 1.1 * dg * du + \
        8 * 2.0 ** -23 * (s * u).abs() + 1e-36


@pytest.mark.parametrize("n_tok", [1, 2, 7, 8, 16, 17, 24, 25, 32, 33, 70])
@pytest.mark.parametrize("d_out,d_in", [(6144, 2048), (7001, 512), (30000, 256), (40, 768), (8, 256),
                                        (10301, 2304), (150001, 256), (80000, 768), (5201, 12544),
                                        (40, 28672)])
def test_gemv_fp4(n_tok, d_out, d_in):
    """One and several passes over the tokens, one and several tiles a CTA, rows
    that end inside a unit, one panel and several, K in one part and in two
    (5201).  (The smaller ones run on either kernel.)"""
    assert fp4(n_tok, d_out, d_in) or d_out * d_in < 2 ** 24
    assert not fp4(1, 40, d_in)
    w = weights((d_out, d_in), d_out + d_in)
    for xt, yt in ((BF16, F32), (F32, BF16), (BF16, BF16), (F32, F32)):
        x = acts(n_tok, d_in, xt, n_tok)
        y = torch.full((n_tok, d_out), 7.0, dtype=yt, device=DEV)
        B.nvfp4_gemv(x, *w, y)
        close(y, *sums_fp4(x, w))


@pytest.mark.parametrize("n_tok", [1, 5, 24, 25, 49])
@pytest.mark.parametrize("d_out,d_in", [(6144, 1024), (20011, 256), (100, 512),
                                        (9505, 2048), (100003, 256), (2605, 12544)])
def test_gemv_swiglu_fp4(n_tok, d_out, d_in):
    assert fp4(n_tok, d_out, d_in, 0, True) or d_out * d_in < 2 ** 24
    gate, up = weights((d_out, d_in), 1 + d_in), weights((d_out, d_in), 2 + d_in)
    for xt in (BF16, F32):
        x = acts(n_tok, d_in, xt, n_tok) * 0.1
        y = torch.full((n_tok, d_out), 7.0, dtype=xt, device=DEV)
        B.nvfp4_gemv_swiglu(x, gate, up, y)
        close(y, *gated_fp4(x, gate, up))


@pytest.mark.parametrize("times", [1, 600])
def test_fp4_bf16_entries_near_their_block_are_exact(times):
    """Entries within 2^-14 of their block's largest lose nothing: one nonzero
    weight a column picks single entries out exactly."""
    d_in = d_out = 256
    assert fp4(4, d_out * times, d_in) == (times > 1)
    g = torch.Generator().manual_seed(1)
    x = (torch.rand((4, d_in), generator=g) + 1) * 2.0 ** -torch.randint(0, 14, (4, d_in), generator=g)
    x = (x * (torch.randint(0, 2, (4, d_in), generator=g) * 2 - 1)).to(BF16).to(DEV)
    x[:, ::16] = 1.5   # (the largest lies in [1, 2) of every block)
    codes = torch.zeros((d_out, d_in), dtype=torch.uint8)
    codes[torch.arange(d_out), torch.arange(d_in)] = 2          # 1.0
    packed = (codes[:, 0::2] | codes[:, 1::2] << 4).to(DEV)
    scales = torch.full((d_out, d_in // 16), 56, dtype=torch.uint8, device=DEV)   # 1.0
    y = torch.empty((4, d_out * times), device=DEV)
    B.nvfp4_gemv(x, packed.repeat(times, 1), scales.repeat(times, 1), torch.ones(1, device=DEV), y)
    assert torch.equal(y, x.float().repeat(1, times))


@pytest.mark.parametrize("d_out", [6200, 40003])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_fp4_extreme_and_nonfinite_tokens(xt, d_out):
    d_in = 512
    assert fp4(9, d_out, d_in) == (d_out > 6200)
    w = weights((d_out, d_in), 3)
    x = acts(9, d_in, F32, 4)
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3, :256] *= 1e-9            # blocks far below the token's largest
    x[4] = 0
    x = x.to(xt)
    x[5, 3], x[6, 400], x[6, 9] = float("nan"), float("inf"), 1.0
    x[7] = 2.0 ** -126
    y = torch.empty((9, d_out), device=DEV)
    B.nvfp4_gemv(x, *w, y)
    keep = [0, 1, 2, 3, 4, 7, 8]
    ref, tol = sums_fp4(x[keep], w)
    assert ((y[keep].double() - ref).abs() <= tol + 2.0 ** -23 * ref.abs() + 2.0 ** -148).all()
    bad = (x[5:7].double()[:, None, :] * dequantised(*w)[None]).sum(-1)
    assert torch.equal(torch.isnan(y[5:7]), torch.isnan(bad))
    inf = torch.isinf(bad)
    assert inf.any() and torch.equal(y[5:7][inf].double(), bad[inf])


FP4_COUNTS = [[1] * 40, [0, 16, 0, 17, 0, 0, 33, 1] * 5, [200], [3, 0, 5, 1, 1, 2, 0, 4] * 16]


@pytest.mark.parametrize("counts", FP4_COUNTS)
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_experts_fp4(counts, pair, xt):
    """Pieces of several experts a CTA and several CTAs an expert, more rows than
    a pass holds, rows behind the last expert's left as they were."""
    E, n, d_in = len(counts), sum(counts), 512
    d_out = max(200, -(-48000000 // (min(E, n) * d_in // 2)) // 8 * 8 + 13)
    n_rows = n + 3
    assert fp4(n_rows, d_out, d_in, E, pair)
    ws_ = [weights((E, d_out, d_in), s) for s in ((5, 6) if pair else (5,))]
    x = acts(50, d_in, xt, 9) * 0.1
    rows = torch.randint(0, 50, (n_rows,), dtype=torch.int32, device=DEV)
    rows[0], rows[n // 2] = -1, 50    # read as rows of zeros
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    y = torch.full((n_rows, d_out), 7.0, dtype=xt, device=DEV)
    if pair:
        B.nvfp4_gemv_swiglu_experts(x, offsets, ws_[0], ws_[1], y, rows)
    else:
        B.nvfp4_gemv_experts(x, offsets, *ws_[0], y, rows)
    bad = (rows < 0) | (rows >= 50)
    xr = torch.where(bad[:, None], torch.zeros((), dtype=xt, device=DEV),
                     x[rows.clamp(0, 49).long()])
    fn = gated_fp4 if pair else sums_fp4
    by_expert(lambda r, *m: close(y[r], *fn(xr[r], *m)), offsets, *ws_)
    assert (y[n:] == 7).all()


def test_fp4_bad_offsets_are_cut():
    E, d_in = 3, 1024
    d_out = 40000
    assert fp4(4, d_out, d_in, E)
    w, x = weights((E, d_out, d_in), 1), acts(4, d_in, BF16, 1)
    y = torch.full((4, d_out), 7.0, device=DEV)
    for offsets, mine in (([-5, 2, 2, 99], {0: 0, 1: 0, 2: 2, 3: 2}), ([3, 1, 2, 2], {1: 1}),
                          ([0, 0, 0, 0], {})):
        y.fill_(7)
        B.nvfp4_gemv_experts(x, torch.tensor(offsets, dtype=torch.int32, device=DEV), *w, y)
        for r in range(4):
            if r in mine:
                e = mine[r]
                close(y[r:r + 1], *sums_fp4(x[r:r + 1], (w[0][e], w[1][e], w[2][e])))
            else:
                assert (y[r] == 7).all()


def test_fp4_unaligned_bases_run_elsewhere():
    """Codes 8 bytes or scales one byte off a 16-byte boundary: same answer."""
    d_out, d_in = 40003, 512
    assert fp4(3, d_out, d_in)
    w, x = weights((d_out, d_in), 8), acts(3, d_in, BF16, 2)
    codes = torch.empty(w[0].numel() + 8, dtype=torch.uint8, device=DEV)[8:].view(w[0].shape)
    scales = torch.empty(w[1].numel() + 1, dtype=torch.uint8, device=DEV)[1:].view(w[1].shape)
    codes.copy_(w[0])
    scales.copy_(w[1])
    for c, s in ((codes, w[1]), (w[0], scales), (w[0], w[1])):
        ws = B.workspace(B.nvfp4_gemv_workspace_size(3, d_out, d_in), DEV)
        ws[:4] = 255
        y = torch.empty((3, d_out), device=DEV)
        B.nvfp4_gemv(x, c, s, w[2], y, ws)
        close(y, *sums_fp4(x, w))
        assert B.nvfp4_workspace_status(ws) == 0


def test_fp4_same_bits_on_streams_and_in_graphs():
    d_out, d_in = 20003, 1024
    assert fp4(6, d_out, d_in)
    w, x = weights((d_out, d_in), 31), acts(6, d_in, BF16, 3)
    y, z, v = (torch.empty((6, d_out), device=DEV) for _ in range(3))
    ws = [B.workspace(B.nvfp4_gemv_workspace_size(6, d_out, d_in), DEV) for _ in range(2)]
    B.nvfp4_gemv(x, *w, y, ws[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.nvfp4_gemv(x, *w, z, ws[0])
        B.nvfp4_gemv(x, *w, z)            # a workspace from the graph's pool
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    z.zero_()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graph.replay()
        B.nvfp4_gemv(x, *w, v, ws[1], stream=side)
        B.nvfp4_gemv(x, *w, v, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, z) and torch.equal(y, v)


@pytest.mark.parametrize("d_out,d_in", [(20003, 1024), (5201, 12544)])
def test_fp4_timeout_is_reported_and_the_context_survives(d_out, d_in):
    """With a wait limit of 1 ns every wait of the kernel gives up: the status
    says so, and the next call is right again."""
    assert fp4(5, d_out, d_in)
    w, x = weights((d_out, d_in), 5), acts(5, d_in, BF16, 3)
    y = torch.zeros((5, d_out), device=DEV)
    ws = B.workspace(B.nvfp4_gemv_workspace_size(5, d_out, d_in), DEV)
    torch.cuda.synchronize()
    B.nvfp4_set_wait_limit_ns(1)
    try:
        B.nvfp4_gemv(x, *w, y, ws)
        torch.cuda.synchronize()
    finally:
        B.nvfp4_set_wait_limit_ns(0)
    assert B.nvfp4_workspace_status(ws) == 6
    B.nvfp4_gemv(x, *w, y, ws)
    assert B.nvfp4_workspace_status(ws) == 0
    close(y, *sums_fp4(x, w))


def test_debug_build_answers_like_the_release_build(monkeypatch):
    """The debug build leaves out pieces of work that are not inside the call's
    arrays; none is, so its results are the release build's, bit for bit."""
    x = acts(40, 1024, BF16, 91)
    w = weights((6200, 1024), 92)
    counts = [0, 5, 1, 0, 33, 20]
    ne = len(counts)
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
    xe = acts(sum(counts), 1024, BF16, 93)
    gate, up = weights((ne, 4352, 1024), 94), weights((ne, 4352, 1024), 95)
    assert fp4(40, 6200, 1024) and fp4(sum(counts), 4352, 1024, ne, True)

    def run():
        y = torch.empty((40, 6200), dtype=BF16, device=DEV)
        z = torch.empty((sum(counts), 4352), dtype=F32, device=DEV)
        for fn, args, size in (
                (B.nvfp4_gemv, (x, *w, y), B.nvfp4_gemv_workspace_size(40, 6200, 1024)),
                (B.nvfp4_gemv_swiglu_experts, (xe, offsets, gate, up, z, None),
                 B.nvfp4_gemv_workspace_size(sum(counts), 4352, 1024, ne, True))):
            ws = B.workspace(size, DEV)
            fn(*args, ws)
            assert B.nvfp4_workspace_status(ws) == 0
        return y, z

    release = run()
    monkeypatch.setattr(B, "_lib", B.debug_lib())
    debug = run()
    monkeypatch.undo()
    for a, b in zip(release, debug):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d_out,d_in", [(1, 6016), (130, 6160), (1100, 8192), (130, 131072)])
@pytest.mark.parametrize("n_tok", [1, 9, 40])
def test_gemv_of_few_columns_and_long_rows(n_tok, d_out, d_in):
    """K in sixteen slices, some of them short."""
    w = weights((d_out, d_in), d_out + d_in)
    for xt, yt in ((BF16, F32), (F32, F32)):
        x = acts(n_tok, d_in, xt, n_tok)
        y = torch.full((n_tok, d_out), 7.0, dtype=yt, device=DEV)
        B.nvfp4_gemv(x, *w, y)
        close(y, *(sums_fp4 if xt == BF16 else sums)(x, w))


def test_swiglu_and_experts_of_few_columns_and_long_rows():
    gate, up = (weights((130, 8192), s) for s in (3, 4))
    x = acts(11, 8192, BF16, 5) * 0.1
    y = torch.full((11, 130), 7.0, device=DEV)
    B.nvfp4_gemv_swiglu(x, gate, up, y)
    close(y, *gated_fp4(x, gate, up))
    w = weights((3, 130, 8192), 6)
    offsets = torch.tensor([1, 1, 4, 7], dtype=torch.int32, device=DEV)
    z = torch.full((11, 130), 7.0, device=DEV)
    B.nvfp4_gemv_experts(x, offsets, *w, z)
    by_expert(lambda r, *m: close(z[r], *sums_fp4(x[r], *m)), offsets, w)
    assert (z[0] == 7).all() and (z[7:] == 7).all()


def test_fp4_halves_of_k_with_nonfinite_tokens():
    d_out, d_in, n = 5201, 12544, 11
    assert fp4(n, d_out, d_in)
    w, x = weights((d_out, d_in), 7), acts(n, d_in, BF16, 8)
    x[3, 9000], x[4, 5], x[10, 12543] = float("nan"), float("inf"), float("-inf")
    y = torch.empty((n, d_out), device=DEV)
    B.nvfp4_gemv(x, *w, y)
    bad = [3, 4, 10]
    keep = [t for t in range(n) if t not in bad]
    close(y[keep], *sums_fp4(x[keep], w))
    ref = (x[bad].double()[:, None, :] * dequantised(*w)[None]).sum(-1)
    assert torch.equal(torch.isnan(y[bad]), torch.isnan(ref))
    inf = torch.isinf(ref)
    assert inf.any() and torch.equal(y[bad][inf].double(), ref[inf])


@pytest.mark.parametrize("counts", [[1, 0, 3, 17, 0, 2, 1, 9], [40, 17, 33, 0, 64, 2, 1, 16]])
@pytest.mark.parametrize("pair,d_out", [(True, 1000), (False, 1004)])
def test_fp4_halves_of_k_by_expert(counts, pair, d_out):
    """One tile a pair of CTAs, and several pieces of several tiles."""
    E, n, d_in = len(counts), sum(counts), 8192 if pair else 16384
    assert fp4(n, d_out, d_in, E, pair)
    ws_ = [weights((E, d_out, d_in), s) for s in ((15, 16) if pair else (15,))]
    x = acts(n, d_in, BF16, 19) * 0.1
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    y = torch.empty((n, d_out), device=DEV)
    ws = B.workspace(B.nvfp4_gemv_workspace_size(n, d_out, d_in, E, pair), DEV)
    if pair:
        B.nvfp4_gemv_swiglu_experts(x, offsets, *ws_, y, None, ws)
    else:
        B.nvfp4_gemv_experts(x, offsets, *ws_[0], y, None, ws)
    assert B.nvfp4_workspace_status(ws) == 0
    fn = gated_fp4 if pair else sums_fp4
    by_expert(lambda r, *m: close(y[r], *fn(x[r], *m)), offsets, *ws_)
