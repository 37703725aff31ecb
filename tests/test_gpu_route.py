"""Tokens sorted by expert and back (nvfp4_moe_sort, _gather, _combine and its
gradient), and a solved mixture-of-experts layer that answers, against plain
implementations.

Tolerances: the sort and the gather are exact.  The weighted sums take k fp32
roundings, each half a step (2^-24) of the sum of absolute values, then one of
the output's type; the dot products d / 32 + 40 of them at most (a lane's
share, then the joins).
"""
import numpy as np
import pytest
import torch

from nvfp4_post_weight_b200 import binding as B
from nvfp4_post_weight_b200.decoder import MoELayerSolver
from test_gpu_gemv import BF16, DEV, F32, acts, close, gated, half_step, sums

pytestmark = pytest.mark.gpu


def routed(T, k, E, seed, dropped=0.2, dtype=np.int32):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, max(E, 1), (T, k))
    gone = rng.random((T, k)) < dropped
    return np.where(gone, rng.choice([-1, E, E + 7, -2 ** 31], (T, k)), ids).astype(dtype)


def sort_plain(ids, E):
    flat = ids.reshape(-1)
    kept = [(e, s) for s, e in enumerate(flat) if 0 <= e < E]
    kept.sort()
    position = np.full(flat.size, -1, np.int32)
    rows = np.full(flat.size, -1, np.int32)
    for r, (_, s) in enumerate(kept):
        position[s], rows[r] = r, s // ids.shape[1]
    offsets = np.searchsorted([e for e, _ in kept], np.arange(E + 1)).astype(np.int32)
    return offsets, rows, position.reshape(ids.shape)


def sort(ids, E, fill=99):
    T, k = ids.shape
    out = (torch.full((E + 1,), fill, dtype=torch.int32, device=DEV),
           torch.full((T * k,), fill, dtype=torch.int32, device=DEV),
           torch.full((T, k), fill, dtype=torch.int32, device=DEV))
    B.nvfp4_moe_sort(torch.from_numpy(ids).to(DEV), *out)
    return out


SORTS = [(1, 1, 1), (1, 8, 128), (7, 3, 5), (64, 8, 128), (33, 2, 1024), (513, 1, 2), (1000, 8, 160),
         (1023, 8, 128), (1024, 8, 128), (1025, 8, 1024), (4099, 6, 31), (8192, 8, 128),
         (8193, 8, 1024), (65537, 1, 700), (65536, 8, 128)]


@pytest.mark.parametrize("T,k,E", SORTS)
@pytest.mark.parametrize("dtype", [np.int32, np.int64])
def test_sort(T, k, E, dtype):
    ids = routed(T, k, E, T + E, dtype=dtype)
    for got, ref in zip(sort(ids, E), sort_plain(ids, E)):
        np.testing.assert_array_equal(got.cpu().numpy(), ref)


def test_sort_extremes():
    for ids, E in ((np.full((70, 4), 3, np.int32), 6),              # one expert has all
                   (np.full((3000, 4), 5, np.int32), 6),            # the last, several CTAs
                   (np.full((3000, 4), -1, np.int32), 6),           # no slot has an expert
                   (np.full((50, 2), 0, np.int32), 0),              # no experts
                   (np.array([[2 ** 40, 1], [-2 ** 40, 2 ** 32]], np.int64), 3),
                   (np.zeros((0, 8), np.int32), 5)):
        for got, ref in zip(sort(ids, E), sort_plain(ids, E)):
            np.testing.assert_array_equal(got.cpu().numpy(), ref)


def test_sort_long_chunks():
    """So many slots that a CTA takes more than the least number of them."""
    rng = np.random.default_rng(0)
    ids = rng.integers(-1, 40, (2 ** 18 + 3, 9)).astype(np.int32)
    E = 40
    offsets, rows, position = (t.cpu().numpy() for t in sort(ids, E))
    flat = ids.reshape(-1)
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    kept = int((flat >= 0).sum())
    np.testing.assert_array_equal(offsets, np.concatenate(
        [[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=E))]))
    np.testing.assert_array_equal(rows[:kept], order[:kept] // 9)
    assert (rows[kept:] == -1).all()
    np.testing.assert_array_equal(position.reshape(-1)[order[:kept]], np.arange(kept))
    assert (position.reshape(-1)[flat < 0] == -1).all()


ROWS = [(1, 1, 1), (1, 8, 4096), (5, 3, 7), (64, 8, 520), (33, 2, 1002), (100, 6, 4104), (9, 9, 16)]


def slots(T, k, seed):
    return sort_plain(routed(T, k, 12, seed), 12)[2]


@pytest.mark.parametrize("T,k,d", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gather_and_its_gradient(T, k, d, dtype):
    pos = slots(T, k, T + d)
    position = torch.from_numpy(pos).to(DEV)
    x = acts(T, d, dtype, 1)
    xs = torch.full((T * k, d), 7.0, dtype=dtype, device=DEV)
    B.nvfp4_moe_gather(x, position, xs)
    ref = torch.full((T * k, d), 7.0, dtype=dtype, device=DEV)
    t, j = np.nonzero(pos >= 0)
    ref[torch.from_numpy(pos[t, j]).long().to(DEV)] = x[torch.from_numpy(t).to(DEV)]
    assert torch.equal(xs, ref)
    # the gradient: the rows' sum back at the tokens
    g = acts(T * k, d, dtype, 2)
    dx = torch.full((T, d), 7.0, dtype=dtype, device=DEV)
    B.nvfp4_moe_combine(g, position, dx)
    close(dx, *combined(g, pos, np.ones(pos.shape)))


def combined(ys, pos, w):
    """(sum, tolerance) in fp64."""
    T, k = pos.shape
    ref = torch.zeros((T, ys.shape[1]), dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(ref)
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                v = ys[pos[t, j]].double() * float(w[t, j])
                ref[t] += v
                mag[t] += v.abs()
    return ref, 2 * k * 2.0 ** -24 * mag


@pytest.mark.parametrize("T,k,d", ROWS)
@pytest.mark.parametrize("st,yt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_combine(T, k, d, st, yt):
    pos = slots(T, k, T + d)
    ys, w = acts(T * k, d, st, 3), torch.rand((T, k), device=DEV)
    y = torch.full((T, d), 7.0, dtype=yt, device=DEV)
    B.nvfp4_moe_combine(ys, torch.from_numpy(pos).to(DEV), y, w)
    close(y, *combined(ys, pos, w.cpu().numpy()))


@pytest.mark.parametrize("T,k,d", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_combine_backward_formula(T, k, d, dtype):
    pos = slots(T, k, T + d)
    position = torch.from_numpy(pos).to(DEV)
    ys, dy, w = acts(T * k, d, dtype, 3), acts(T, d, dtype, 4), torch.rand((T, k), device=DEV)
    dys = torch.full((T * k, d), 7.0, dtype=dtype, device=DEV)
    dw = torch.full((T, k), 7.0, device=DEV)
    B.nvfp4_moe_combine_backward(dy, ys, position, w, dys, dw)
    named = np.zeros(T * k, bool)
    for t in range(T):
        for j in range(k):
            p = pos[t, j]
            if p < 0:
                assert dw[t, j] == 0
                continue
            named[p] = True
            ref = dy[t].double() * w[t, j].double()
            assert ((dys[p].double() - ref).abs() <= 1.01 * (half_step(dtype) + 2.0 ** -24) * ref.abs()
                    + 1e-38).all()
            dot = dy[t].double() * ys[p].double()
            assert abs(dw[t, j].item() - dot.sum().item()) <= \
                (d / 32 + 40) * 2.0 ** -24 * dot.abs().sum().item()
    assert (dys[torch.from_numpy(~named).to(DEV)] == 7).all()


def test_gradients_against_differences():
    """<dL/dYs, v> and <dL/dw, u> by differences of L = <G, combine(Ys, w)>,
    which is bilinear: central differences are exact up to rounding (fp32:
    each L sums T d terms of k roundings; 1e-4 of the terms' absolute sum is
    far above (k + log) 2^-24 / step with a step of 1)."""
    T, k, d = 12, 4, 40
    pos = torch.from_numpy(slots(T, k, 5)).to(DEV)
    ys, G, w = acts(T * k, d, F32, 1), acts(T, d, F32, 2), torch.rand((T, k), device=DEV)
    v, u = acts(T * k, d, F32, 3), torch.randn((T, k), device=DEV)

    def loss(ys, w):
        y = torch.empty((T, d), device=DEV)
        B.nvfp4_moe_combine(ys.contiguous(), pos, y, w.contiguous())
        return (G.double() * y.double()).sum().item()

    dys, dw = torch.zeros_like(ys), torch.empty((T, k), device=DEV)
    B.nvfp4_moe_combine_backward(G, ys, pos, w, dys, dw)
    size = (G.abs().double().sum() * (ys.abs().max() + v.abs().max())).item()
    assert abs((loss(ys + v, w) - loss(ys - v, w)) / 2 - (dys.double() * v.double()).sum().item()) \
        <= 1e-4 * size
    assert abs((loss(ys, w + u) - loss(ys, w - u)) / 2 - (dw.double() * u.double()).sum().item()) \
        <= 1e-4 * size


def test_rows_without_a_slot_and_bad_positions():
    """Masked slots add nothing even where a weight or a row is not finite; a
    position outside the rows names none."""
    ys = torch.full((6, 16), float("nan"), device=DEV)
    ys[2] = 3.0
    pos = torch.tensor([[-1, 2], [-1, -1], [6, 2 ** 31 - 1]], dtype=torch.int32, device=DEV)
    w = torch.full((3, 2), float("inf"), device=DEV)
    w[0, 1] = 0.5
    y = torch.full((3, 16), 7.0, device=DEV)
    B.nvfp4_moe_combine(ys, pos, y, w)
    assert (y[0] == 1.5).all() and (y[1:] == 0).all()
    x = acts(3, 16, F32, 1)
    xs = torch.full((6, 16), 7.0, device=DEV)
    B.nvfp4_moe_gather(x, pos, xs)
    assert torch.equal(xs[2], x[0]) and (xs[[0, 1, 3, 4, 5]] == 7).all()
    dys, dw = torch.full((6, 16), 7.0, device=DEV), torch.full((3, 2), 7.0, device=DEV)
    B.nvfp4_moe_combine_backward(x, ys, pos, w, dys, dw)
    assert torch.equal(dys[2], 0.5 * x[0]) and (dys[[0, 1, 3, 4, 5]] == 7).all()
    assert (dw.reshape(-1)[[0, 2, 3, 4, 5]] == 0).all() and dw[0, 1] != 0


def test_odd_bases():
    """Rows that start off every vector boundary."""
    T, k, d = 5, 2, 64
    pos = torch.from_numpy(slots(T, k, 3)).to(DEV)

    def odd(t):
        return torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape).copy_(t)

    x, ys, w = acts(T, d, BF16, 1), acts(T * k, d, BF16, 2), torch.rand((T, k), device=DEV)
    outs = []
    for f in (lambda t: t, odd):
        xs, y = f(torch.zeros((T * k, d), dtype=BF16, device=DEV)), \
            f(torch.zeros((T, d), dtype=BF16, device=DEV))
        dys, dw = f(torch.zeros_like(ys)), f(torch.zeros((T, k), device=DEV))
        B.nvfp4_moe_gather(f(x), pos, xs)
        B.nvfp4_moe_combine(f(ys), pos, y, f(w))
        B.nvfp4_moe_combine_backward(f(x), f(ys), pos, f(w), dys, dw)
        outs.append((xs, y, dys, dw))
    for a, b in zip(*outs):
        assert (a.float() - b.float()).abs().max() <= 1e-4 * a.float().abs().max()
    assert torch.equal(outs[0][0], outs[1][0])


# ---- a solved layer, together ------------------------------------------------------
def solved_layer():
    E, hidden, inter, T, k = 6, 64, 48, 200, 2
    s = MoELayerSolver(E, hidden, inter, DEV)
    g = torch.Generator().manual_seed(3)
    Ws = [(torch.randn(shape, generator=g) * 0.1).to(BF16).to(DEV) for shape in s.wshape]
    X = acts(T, hidden, BF16, 4)
    ids = torch.from_numpy(routed(T, k, E, 5, dropped=0.05)).to(DEV)
    return s, Ws, X, ids


def expert(stacked, e):
    return tuple(t[e:e + 1] if t.dim() == 1 else t[e] for t in stacked)


def test_moe_layer_from_routing_to_answer():
    """Calibration tokens by expert into the batched Hessians, the solve, and
    the answer of the solved layer for a padded batch, on a stream of its own
    and captured."""
    s, Ws, X, ids = solved_layer()
    Xin = s.tokens_by_expert(X, ids)
    for e in range(s.E):
        t = torch.nonzero((ids == e))[:, 0]
        assert torch.equal(Xin[e], X[t])
    Xmid = [torch.nn.functional.silu(x.float() @ Ws[3 * e].float().T) *
            (x.float() @ Ws[3 * e + 1].float().T) for e, x in enumerate(Xin)]
    Xs = [t for e in range(s.E) for t in (Xin[e], Xmid[e].to(BF16))]
    s.step(Ws, Xs)
    assert s.status() == (0, 0, 0, 0)
    # the lists are views of the stacked results
    assert torch.equal(s.codes[4], s.stacked["up"][0][1])
    assert s.s_g[5].item() == s.stacked["down"][2][1].item()

    x, few = X[:9].clone(), ids[:9].clone()
    few[3] = -1
    w = torch.softmax(torch.randn((9, 2), device=DEV), 1)

    def check(y):
        mid, ref = {}, torch.zeros((9, s.hidden), dtype=torch.float64, device=DEV)
        tol = torch.zeros_like(ref)
        for t in range(9):
            for j in range(2):
                e = int(few[t, j])
                if not 0 <= e < s.E:
                    continue
                h, dh = gated(x[t:t + 1], expert(s.stacked["gate"], e), expert(s.stacked["up"], e))
                q = expert(s.stacked["down"], e)
                v, dv = sums(h, q)
                # the intermediate's tolerance and its rounding to bf16 through |Q|
                _, mag = sums(dh + half_step(BF16) * (h.abs() + dh), q)
                n = mag / ((s.inter / 32 + 160) * 2.0 ** -23)
                wt = w[t, j].double()
                ref[t] += wt * v[0]
                tol[t] += wt * (dv + n + 4 * 2.0 ** -24 * (v.abs() + dv + n))[0]
        close(y, ref, tol)

    y = s.forward(x, few, w)
    assert (y[3] == 0).all()
    check(y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = s.forward(x, few, w, stream=side)
    side.synchronize()
    assert torch.equal(y, y2)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(x)
    with torch.cuda.graph(graph):
        s.forward(x, few, w, out)
    x.copy_(X[20:29])
    few.copy_(ids[30:39])
    graph.replay()
    torch.cuda.synchronize()
    check(out)


def test_two_graphs_and_an_eager_call_side_by_side():
    """No state is kept between calls: two captured sorts replayed on two
    streams beside an eager one."""
    a, b, c = (routed(3000, 8, 128, s) for s in (1, 2, 3))
    outs, graphs, ins = [], [], []
    for ids in (a, b):
        t = torch.from_numpy(ids).to(DEV)
        out = sort(ids, 128)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.nvfp4_moe_sort(t, *out)
        for o in out:
            o.fill_(0)
        outs.append(out)
        graphs.append(g)
        ins.append(t)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for g, st in zip(graphs, streams):
        with torch.cuda.stream(st):
            g.replay()
    out_c = sort(c, 128)
    torch.cuda.synchronize()
    for out, ids in zip((*outs, out_c), (a, b, c)):
        for got, ref in zip(out, sort_plain(ids, 128)):
            np.testing.assert_array_equal(got.cpu().numpy(), ref)
