"""Refusals of the products with solved weights and of the routing calls: the
library's host-side checks (no device is touched) and the binding's."""
import ctypes

import pytest
import torch

from nvfp4_post_weight_b200 import binding as B

P = ctypes.c_void_p
OK, ARG, SHAPE = 0, 1, 2
A = P(256)


def gemv(X=A, xt=0, n=1, c=A, s=A, g=A, o=16, i=32, Y=A, yt=0, ws=None, nws=0):
    return B.lib().nvfp4_gemv(X, xt, n, c, s, g, o, i, Y, yt, ws, nws, None)


def experts(X=A, xt=0, n_x=4, rows=A, off=A, E=2, n=4, c=A, s=A, g=A, o=16, i=32, Y=A, yt=0):
    return B.lib().nvfp4_gemv_experts(X, xt, n_x, rows, off, E, n, c, s, g, o, i, Y, yt, None, 0,
                                      None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), ARG), (dict(o=-1), ARG), (dict(i=-16), ARG), (dict(xt=2), ARG), (dict(yt=-1), ARG),
    (dict(X=None), ARG), (dict(c=None), ARG), (dict(s=None), ARG), (dict(g=None), ARG),
    (dict(Y=None), ARG), (dict(X=P(264)), ARG), (dict(c=P(260)), ARG), (dict(Y=P(257)), ARG),
    (dict(Y=P(258), yt=1), ARG), (dict(i=24), SHAPE), (dict(i=(1 << 17) + 16), SHAPE),
    (dict(o=(1 << 22) + 1), SHAPE), (dict(n=(1 << 22) + 1), SHAPE),
    (dict(n=0), OK), (dict(o=0), OK), (dict(n=0, X=None, Y=None, c=None, s=None, g=None), OK)])
def test_gemv_refuses(kw, status):
    assert gemv(**kw) == status


def test_gemv_swiglu_refuses():
    f = B.lib().nvfp4_gemv_swiglu
    assert f(A, 0, 1, A, A, A, None, A, A, 16, 32, A, 0, None, 0, None) == ARG
    assert f(A, 0, 1, A, A, A, A, A, None, 16, 32, A, 0, None, 0, None) == ARG
    assert f(A, 0, 1, A, A, A, P(260), A, A, 16, 32, A, 0, None, 0, None) == ARG
    assert f(A, 0, 1, A, A, A, A, A, A, 16, 40, A, 0, None, 0, None) == SHAPE
    assert f(A, 0, 0, A, A, A, A, A, A, 16, 32, A, 0, None, 0, None) == OK


def test_gemv_refuses_a_missing_or_small_workspace():
    o = 40003
    need = B.nvfp4_gemv_workspace_size(3, o, 512)
    assert need > 3 * 512 * 4 and B.nvfp4_gemv_workspace_size(3, 16, 512) == 0
    assert B.nvfp4_gemv_workspace_size(3, o, 528) == 0
    assert B.nvfp4_gemv_workspace_size(3, o, 1 << 40) == 0
    assert B.nvfp4_gemv_workspace_size(3, 1 << 40, 512) == 0
    assert B.lib().nvfp4_gemv_workspace_size(-1, o, 512, 0, 0, 0) == 0
    assert B.nvfp4_gemv_workspace_size(3, o, 512, dtype=torch.float32) == 0
    for kw in (dict(), dict(ws=A, nws=need - 1), dict(ws=P(128), nws=need)):
        assert gemv(n=3, o=o, i=512, **kw) == 3
    assert gemv(n=0, o=o, i=512) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(off=None), ARG), (dict(rows=None, n_x=3), ARG), (dict(n_x=-1), ARG), (dict(E=-1), ARG),
    (dict(rows=P(258)), ARG), (dict(off=P(257)), ARG), (dict(E=1025), SHAPE),
    (dict(n=(1 << 22) + 1), SHAPE), (dict(n_x=(1 << 22) + 1), SHAPE), (dict(X=None), ARG),
    (dict(E=0), OK), (dict(n=0), OK)])
def test_gemv_experts_refuses(kw, status):
    assert experts(**kw) == status
    L = B.lib()
    d = dict(X=A, xt=0, n_x=4, rows=A, off=A, E=2, n=4, o=16, i=32, Y=A, yt=0)
    d.update(kw)
    assert L.nvfp4_gemv_swiglu_experts(d["X"], d["xt"], d["n_x"], d["rows"], d["off"], d["E"],
                                       d["n"], A, A, A, A, A, A, d["o"], d["i"], d["Y"], d["yt"],
                                       None, 0, None) == status


def test_routing_calls_refuse():
    L = B.lib()
    big = 1 << 26

    def sort(ids=A, nb=4, n=4, k=2, E=8, off=A, rows=A, pos=A):
        return L.nvfp4_moe_sort(ids, nb, n, k, E, off, rows, pos, None)

    for kw, status in ((dict(ids=None), ARG), (dict(nb=2), ARG), (dict(n=-1), ARG), (dict(k=0), ARG),
                       (dict(E=-1), ARG), (dict(off=None), ARG), (dict(rows=None), ARG),
                       (dict(pos=None), ARG), (dict(E=1025), SHAPE), (dict(k=1025), SHAPE),
                       (dict(n=big + 1), SHAPE), (dict(n=big, k=17), SHAPE),
                       (dict(ids=P(260), nb=8), ARG), (dict(rows=P(258)), ARG)):
        assert sort(**kw) == status, kw

    def gather(X=A, dt=0, pos=A, n=4, k=2, d=8, Xs=A):
        return L.nvfp4_moe_gather(X, dt, pos, n, k, d, Xs, None)

    for kw, status in ((dict(X=None), ARG), (dict(dt=3), ARG), (dict(pos=None), ARG),
                       (dict(Xs=None), ARG), (dict(d=-1), ARG), (dict(d=(1 << 17) + 1), SHAPE),
                       (dict(k=0), ARG), (dict(X=P(257)), ARG), (dict(X=P(258), dt=1), ARG),
                       (dict(n=0), OK), (dict(d=0), OK)):
        assert gather(**kw) == status, kw

    def combine(Ys=A, st=0, pos=A, w=A, n=4, k=2, d=8, Y=A, yt=0):
        return L.nvfp4_moe_combine(Ys, st, pos, w, n, k, d, Y, yt, None)

    for kw, status in ((dict(Ys=None), ARG), (dict(st=3), ARG), (dict(yt=3), ARG),
                       (dict(pos=None), ARG), (dict(Y=None), ARG), (dict(w=P(258)), ARG),
                       (dict(n=big, k=17), SHAPE), (dict(n=0), OK)):
        assert combine(**kw) == status, kw

    def backward(dY=A, Ys=A, dt=0, pos=A, w=A, n=4, k=2, d=8, dYs=A, dw=A):
        return L.nvfp4_moe_combine_backward(dY, Ys, dt, pos, w, n, k, d, dYs, dw, None)

    for kw, status in ((dict(dY=None), ARG), (dict(Ys=None), ARG), (dict(w=None), ARG),
                       (dict(dYs=None), ARG), (dict(dw=None), ARG), (dict(dt=2), ARG),
                       (dict(dYs=P(257)), ARG), (dict(n=-1), ARG), (dict(n=0), OK)):
        assert backward(**kw) == status, kw


def test_binding_refuses_host_tensors():
    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    x, y = torch.zeros((1, 32), dtype=bf), torch.zeros((1, 16), dtype=bf)
    w = (torch.zeros((16, 16), dtype=u8), torch.zeros((16, 2), dtype=u8), torch.zeros(1))
    off, pos = torch.zeros(3, dtype=i32), torch.zeros((1, 2), dtype=i32)
    for call in (lambda: B.nvfp4_gemv(x, *w, y),
                 lambda: B.nvfp4_gemv_swiglu(x, w, w, y),
                 lambda: B.nvfp4_gemv_experts(x, off, *w, y),
                 lambda: B.nvfp4_gemv_experts(x, None, *w, y),
                 lambda: B.nvfp4_gemv_swiglu_experts(x, off, w, w, y),
                 lambda: B.nvfp4_moe_sort(pos, off, off, pos),
                 lambda: B.nvfp4_moe_gather(x, pos, x),
                 lambda: B.nvfp4_moe_combine(x, pos, x),
                 lambda: B.nvfp4_moe_combine_backward(x, x, pos, pos, x, pos)):
        with pytest.raises(B.Nvfp4Error) as e:
            call()
        assert e.value.code == ARG


@pytest.mark.gpu
def test_binding_refuses_wrong_shapes_types_and_streams():
    dev, bf, u8, i32 = "cuda:0", torch.bfloat16, torch.uint8, torch.int32

    def z(*shape, dtype=bf):
        return torch.zeros(shape, dtype=dtype, device=dev)

    x, y = z(4, 32), z(4, 16)
    w = (z(16, 16, dtype=u8), z(16, 2, dtype=u8), z(1, dtype=torch.float32))
    we = (z(2, 16, 16, dtype=u8), z(2, 16, 2, dtype=u8), z(2, dtype=torch.float32))
    off, rows, pos = z(3, dtype=i32), z(4, dtype=i32), z(2, 2, dtype=i32)
    f = torch.float32
    bad = [lambda: B.nvfp4_gemv(x, w[0][:8], w[1], w[2], y),
           lambda: B.nvfp4_gemv(x, w[0], w[1][:, :1], w[2], y),
           lambda: B.nvfp4_gemv(x, *w, y[:3]),
           lambda: B.nvfp4_gemv(x, *w, z(4, 16, dtype=torch.float16)),
           lambda: B.nvfp4_gemv(x[:, ::2], *w, y),
           lambda: B.nvfp4_gemv(z(4, 24), z(16, 12, dtype=u8), z(16, 1, dtype=u8), w[2], y),
           lambda: B.nvfp4_gemv_swiglu(x, w, w[:2], y),
           lambda: B.nvfp4_gemv_swiglu(x, w, we, y),
           lambda: B.nvfp4_gemv_experts(x, off, *w, y),
           lambda: B.nvfp4_gemv_experts(x, off.long(), *we, y),
           lambda: B.nvfp4_gemv_experts(x, off, *we, y, rows[:3]),
           lambda: B.nvfp4_gemv_experts(x[:2], off, *we, y),
           lambda: B.nvfp4_moe_sort(pos.float(), off, rows, pos),
           lambda: B.nvfp4_moe_sort(pos, off, rows[:3], pos),
           lambda: B.nvfp4_moe_sort(pos, off, rows, pos.long()),
           lambda: B.nvfp4_moe_gather(x[:2], pos, z(4, 32, dtype=f)),
           lambda: B.nvfp4_moe_gather(x[:2], pos, z(3, 32)),
           lambda: B.nvfp4_moe_gather(x, pos, x),
           lambda: B.nvfp4_moe_combine(x, pos, z(3, 32)),
           lambda: B.nvfp4_moe_combine(x, pos, z(2, 32), z(2, 2)),
           lambda: B.nvfp4_moe_combine_backward(z(2, 32), z(4, 32, dtype=f), pos, z(2, 2, dtype=f),
                                                x, z(2, 2, dtype=f)),
           lambda: B.nvfp4_moe_combine_backward(z(2, 32), x, pos, z(2, 2, dtype=f), x, z(4, dtype=f))]
    for k, call in enumerate(bad):
        with pytest.raises(B.Nvfp4Error):
            call()
            print(k)


class _On:
    """A tensor as the binding's checks see it, on a device of any number."""
    is_cuda, dtype, shape = True, torch.float32, (2,)

    def __init__(self, n):
        self.n, self.device = n, torch.device("cuda", n)

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.n

    def data_ptr(self):
        return 256


def test_a_stream_or_tensor_of_another_device_is_refused(monkeypatch):
    """The device checks come before the library is called; the call itself runs
    with the tensors' device current."""
    monkeypatch.setattr(torch, "Tensor", _On)
    assert B._arg("nvfp4_gemv", _On(1), "Y", (2,), torch.float32, 1) == 256
    with pytest.raises(B.Nvfp4Error, match="tensors on cuda:0 and cuda:1"):
        B._arg("nvfp4_gemv", _On(1), "Y", (2,), torch.float32, 0)
    stream = type("S", (), dict(device=torch.device("cuda", 0), cuda_stream=7))()
    with pytest.raises(B.Nvfp4Error, match="stream of cuda:0, tensors on cuda:1"):
        B._run_on("nvfp4_gemv", 1, stream)
    seen = []

    class device:
        def __init__(self, n):
            self.n = n

        def __enter__(self):
            seen.append(self.n)

        def __exit__(self, *a):
            seen.append("out")

    class L:
        def nvfp4_gemv(self, *a):
            seen.append(a)
            return 0
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(B, "lib", L)
    B._run_on("nvfp4_gemv", 0, stream, 5)
    assert seen == [0, (5, 7), "out"]


def test_no_sorted_rows_need_no_row_indices():
    """An empty array has no address: rows of no entries are as good as any."""
    for f, w in ((B.lib().nvfp4_gemv_experts, (A, A, A)),
                 (B.lib().nvfp4_gemv_swiglu_experts, (A,) * 6)):
        assert f(A, 0, 3, None, A, 2, 0, *w, 16, 32, None, 0, None, 0, None) == OK
        assert f(A, 0, 3, None, A, 2, 1, *w, 16, 32, A, 0, None, 0, None) == ARG


@pytest.mark.parametrize("w", [None, 5, torch.zeros((3, 4)), (None, None)])
def test_a_weight_is_three_tensors(w):
    with pytest.raises(B.Nvfp4Error, match="expected \\(codes, scales, global_scale\\)") as e:
        B._weight("nvfp4_gemv_swiglu", "gate ", w, (), 16, 32, 0)
    assert e.value.code == ARG


# (rows, d_out, d_in, experts, pair): whether the FP4 tensor cores were measured a fifth
# or more faster than the decoding kernel, or slower
PATHS = [((1, 1024, 8192, 0, False), False), ((32, 1024, 8192, 0, False), False),
         ((65, 1024, 8192, 0, False), True), ((96, 1024, 1024, 0, False), True),
         ((96, 256, 1024, 0, False), True), ((32, 256, 1024, 0, False), False),
         ((65, 2048, 2048, 0, False), True), ((2049, 1024, 1024, 0, False), True),
         ((8192, 256, 1024, 0, False), True), ((32, 8192, 8192, 0, False), True),
         ((512, 128, 1024, 512, False), False), ((1024, 128, 1024, 512, False), False),
         ((8192, 128, 1024, 512, False), False), ((32768, 128, 1024, 256, False), False),
         ((4096, 256, 512, 256, True), False), ((16384, 512, 512, 512, False), False),
         ((8192, 128, 128, 1024, False), False), ((8192, 256, 512, 128, False), False),
         ((16384, 64, 512, 64, True), False), ((64, 768, 2048, 8, True), True),
         ((128, 768, 2048, 8, True), True), ((32, 768, 2048, 8, True), False),
         ((128, 2048, 1024, 16, False), True), ((192, 768, 768, 32, True), True),
         ((64, 256, 1024, 64, True), False), ((8192, 768, 2048, 128, True), True),
         ((8, 1536, 4096, 8, True), True), ((1024, 1024, 1024, 1, False), True),
         ((8192, 64, 256, 8, False), True), ((8192, 4096, 2304, 8, False), True)]


@pytest.mark.parametrize("sizes,path", PATHS)
def test_the_faster_kernel_is_chosen(sizes, path):
    assert (B.nvfp4_gemv_workspace_size(*sizes) > 0) == path
