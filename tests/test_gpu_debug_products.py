"""The debug build's products and routing: every index is checked against its array,
none leaves it, and the results are the release build's bit for bit, at odd sizes and
at sizes of every form of the kernels."""
import numpy as np
import pytest
import torch

from nvfp4_post_weight_b200 import binding as B
from test_gpu_gemv import BF16, COUNTS, DEV, F32, SHAPES, acts, weights
from test_gpu_route import ROWS, SORTS, routed, slots, sort

pytestmark = pytest.mark.gpu


def both(monkeypatch, run):
    """run() by the release and by the debug build: equal tensors, no check failed."""
    release = run()
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(B, "_lib", B.debug_lib())
        assert B.lib().nvfp4_debug_build() == 1
        B.nvfp4_product_status()
        debug = run()
        assert B.nvfp4_product_status() == 0
    for a, b in zip(release, debug):
        assert torch.equal(a, b)


MORE = [(9, 6144, 2048), (3, 5201, 12544), (2049, 130, 512), (40, 20003, 1024), (1, 256, 16384),
        (5, 4001, 4112), (33, 40, 28672)]


@pytest.mark.parametrize("n,d_out,d_in", SHAPES + MORE)
def test_products(monkeypatch, n, d_out, d_in):
    w, up = weights((d_out, d_in), 1), weights((d_out, d_in), 2)

    def run():
        out = []
        for xt in (BF16, F32):
            x = acts(n, d_in, xt, 3) * 0.1
            y, z = (torch.full((n, d_out), 7.0, dtype=t, device=DEV) for t in (F32, BF16))
            B.nvfp4_gemv(x, *w, y)
            B.nvfp4_gemv_swiglu(x, w, up, z)
            out += [y, z]
        return out
    both(monkeypatch, run)


@pytest.mark.parametrize("counts", COUNTS + [[5, 2100, 0, 700, 33]])
@pytest.mark.parametrize("d_out,d_in", [(40, 272), (136, 1024), (4001, 1024)])
def test_products_by_expert(monkeypatch, counts, d_out, d_in):
    E, n = len(counts), sum(counts) + 3
    w, up = weights((E, d_out, d_in), 1), weights((E, d_out, d_in), 2)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    rows = torch.randint(-1, 12, (n,), dtype=torch.int32, device=DEV)

    def run():
        out = []
        for xt in (BF16, F32):
            x = acts(11, d_in, xt, 3) * 0.1
            y, z = (torch.full((n, d_out), 7.0, dtype=t, device=DEV) for t in (F32, BF16))
            B.nvfp4_gemv_experts(x, offsets, *w, y, rows)
            B.nvfp4_gemv_swiglu_experts(x, offsets, w, up, z, rows)
            out += [y, z]
        return out
    both(monkeypatch, run)


@pytest.mark.parametrize("T,k,E", SORTS)
def test_sort(monkeypatch, T, k, E):
    ids = routed(T, k, E, T + E)
    both(monkeypatch, lambda: sort(ids, E))


@pytest.mark.parametrize("T,k,d", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows(monkeypatch, T, k, d, dtype):
    position = torch.from_numpy(slots(T, k, T + d)).to(DEV)
    x, ys, w = acts(T, d, dtype, 1), acts(T * k, d, dtype, 2), torch.rand((T, k), device=DEV)

    def run():
        xs, dys = (torch.full((T * k, d), 7.0, dtype=dtype, device=DEV) for _ in range(2))
        y, dw = torch.empty((T, d), dtype=BF16, device=DEV), torch.empty((T, k), device=DEV)
        B.nvfp4_moe_gather(x, position, xs)
        B.nvfp4_moe_combine(ys, position, y, w)
        B.nvfp4_moe_combine_backward(x, ys, position, w, dys, dw)
        return xs, y, dys, dw
    both(monkeypatch, run)
