"""Products of many rows on the block-scaled FP4 tensor cores: rows in several
parts, outputs of few columns, more rows than experts' passes."""
import numpy as np
import pytest
import torch

from nvfp4_post_weight_b200 import binding as B
from test_gpu_gemv import (BF16, DEV, F32, acts, by_expert, close, dequantised, fp4, gated_fp4,
                           sums_fp4, weights)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2048, 2049, 4097, 6001])
@pytest.mark.parametrize("d_out,d_in,yt", [(40, 768, F32), (1025, 1024, BF16)])
def test_rows_in_parts(n, d_out, d_in, yt):
    assert fp4(n, d_out, d_in)
    w, x = weights((d_out, d_in), 1), acts(n, d_in, BF16, 2)
    y = torch.full((n, d_out), 7.0, dtype=yt, device=DEV)
    B.nvfp4_gemv(x, *w, y)
    close(y, *sums_fp4(x, w))
    up = weights((d_out, d_in), 3)
    assert fp4(n, d_out, d_in, 0, True)
    B.nvfp4_gemv_swiglu(x * 0.1, w, up, y)
    close(y, *gated_fp4(x * 0.1, w, up))


@pytest.mark.parametrize("counts", [[0, 700, 0, 2000, 1, 0, 1300, 90], [2048, 1], [5000],
                                    [1000, 1048, 0, 1, 2047]])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("indexed", [False, True])
def test_experts_rows_in_parts(counts, pair, indexed):
    """Parts that end inside an expert's rows, at them and behind the last."""
    E, n, d_in = len(counts), sum(counts), 1024
    d_out = 4700 if E < 3 else 2001
    n_rows = n + 5
    assert fp4(n_rows, d_out, d_in, E, pair)
    ws_ = [weights((E, d_out, d_in), s) for s in ((5, 6) if pair else (5,))]
    x = acts(50 if indexed else n_rows, d_in, BF16, 9) * 0.1
    rows = torch.randint(-1, 51, (n_rows,), dtype=torch.int32, device=DEV) if indexed else None
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    y = torch.full((n_rows, d_out), 7.0, device=DEV)
    if pair:
        B.nvfp4_gemv_swiglu_experts(x, offsets, ws_[0], ws_[1], y, rows)
    else:
        B.nvfp4_gemv_experts(x, offsets, *ws_[0], y, rows)
    xr = x
    if indexed:
        none = ((rows < 0) | (rows >= 50))[:, None]
        xr = torch.where(none, torch.zeros((), dtype=BF16, device=DEV), x[rows.clamp(0, 49).long()])
    fn = gated_fp4 if pair else sums_fp4
    by_expert(lambda r, *m: close(y[r], *fn(xr[r], *m)), offsets, *ws_)
    assert (y[n:] == 7).all()


def test_parts_and_bad_offsets():
    """Offsets outside the rows, far outside and descending, cut in every part."""
    E, n, d_out, d_in = 4, 4500, 2001, 1024
    assert fp4(n, d_out, d_in, E)
    w, x = weights((E, d_out, d_in), 1), acts(n, d_in, BF16, 1)
    offsets = torch.tensor([-2 ** 31, 100, 50, 3000, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    y = torch.full((n, d_out), 7.0, device=DEV)
    B.nvfp4_gemv_experts(x, offsets, *w, y)
    # expert 0: 0..99, expert 1: none, expert 2: 50..2999, expert 3 the rest; rows of
    # two experts get either's answer
    m = [tuple(t[e] for t in w) for e in range(E)]
    close(y[:50], *sums_fp4(x[:50], m[0]))
    close(y[100:3000], *sums_fp4(x[100:3000], m[2]))
    close(y[3000:], *sums_fp4(x[3000:], m[3]))


def test_status_of_all_parts():
    """A workspace serves every part, and its status word begins each call."""
    n, d_out, d_in = 4097, 300, 1024
    size = B.nvfp4_gemv_workspace_size(n, d_out, d_in)
    assert size == B.nvfp4_gemv_workspace_size(2048, d_out, d_in) > 0
    w, x = weights((d_out, d_in), 1), acts(n, d_in, BF16, 2)
    ws = B.workspace(size, DEV)
    ws.fill_(255)
    y = torch.empty((n, d_out), device=DEV)
    B.nvfp4_gemv(x, *w, y, ws)
    assert B.nvfp4_workspace_status(ws) == 0
    close(y, *sums_fp4(x, w))


# outputs narrower than a tile, one unit of eight columns or less, tiles of every size
@pytest.mark.parametrize("d_out", [1, 8, 13, 40, 129, 300])
@pytest.mark.parametrize("n,d_in", [(300, 256), (333, 768), (700, 2048)])
def test_few_columns_of_many_rows(d_out, n, d_in):
    assert fp4(n, d_out, d_in)
    w, x = weights((d_out, d_in), d_out), acts(n, d_in, BF16, 2)
    y = torch.full((n, d_out), 7.0, device=DEV)
    B.nvfp4_gemv(x, *w, y)
    close(y, *sums_fp4(x, w))


@pytest.mark.parametrize("pair", [False, True])
def test_nonfinite_tokens_of_pairs_and_experts(pair):
    """A NaN or an infinity stays in its row and its expert's weights, as in the plain
    product."""
    counts = [3, 0, 17, 1, 33, 8]
    E, n, d_in = len(counts), sum(counts), 512
    d_out = 13007 if not pair else 7001
    assert fp4(n, d_out, d_in, E, pair)
    ws_ = [weights((E, d_out, d_in), s) for s in ((5, 6) if pair else (5,))]
    x = acts(20, d_in, BF16, 9) * 0.1
    x[3, 7], x[5, 500], x[9, 0] = float("nan"), float("inf"), float("-inf")
    rows = torch.arange(n, dtype=torch.int32, device=DEV) * 7 % 20
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    y = torch.full((n, d_out), 7.0, device=DEV)
    if pair:
        B.nvfp4_gemv_swiglu_experts(x, offsets, *ws_, y, rows)
    else:
        B.nvfp4_gemv_experts(x, offsets, *ws_[0], y, rows)
    xr = x[rows.long()]
    bad = ~torch.isfinite(xr.float()).all(1)

    def check(r, *m):
        good = ~bad[r]
        if good.any():
            close(y[r][good], *(gated_fp4 if pair else sums_fp4)(xr[r][good], *m))
        for k in torch.nonzero(bad[r])[:, 0].tolist():
            v = [(xr[r][k].double()[None] * dequantised(*q)).sum(1) for q in m]
            ref = v[0] / (1 + torch.exp(-v[0])) * v[1] if pair else v[0]
            got = y[r][k].double()
            assert torch.equal(torch.isnan(got), torch.isnan(ref))
            inf = torch.isinf(ref)
            assert torch.equal(got[inf], ref[inf])
            assert not (torch.isfinite(ref).any() and not pair)
    by_expert(check, offsets, *ws_)


@pytest.mark.parametrize("E,d_out,n", [(1, 8, 700), (3, 13, 900), (2, 130, 2500)])
@pytest.mark.parametrize("pair", [False, True])
def test_few_experts_of_many_rows(E, d_out, n, pair):
    """Few columns: few CTAs in the general kernel, so the passes go to this one."""
    d_in = 512
    assert fp4(n, d_out, d_in, E, pair)
    ws_ = [weights((E, d_out, d_in), s) for s in ((5, 6) if pair else (5,))]
    x = acts(n, d_in, BF16, 9) * 0.1
    ends = torch.arange(E + 1) * (n - 7) // E
    offsets = (ends + 3).int().to(DEV)      # three rows before the first expert's
    y = torch.full((n, d_out), 7.0, device=DEV)
    if pair:
        B.nvfp4_gemv_swiglu_experts(x, offsets, *ws_, y)
    else:
        B.nvfp4_gemv_experts(x, offsets, *ws_[0], y)
    fn = gated_fp4 if pair else sums_fp4
    by_expert(lambda r, *m: close(y[r], *fn(x[r], *m)), offsets, *ws_)
    assert (y[:3] == 7).all() and (y[n - 4:] == 7).all()
