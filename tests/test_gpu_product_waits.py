"""Timed-out waits of the products on the block-scaled FP4 tensor cores: whatever
role gives up first, no CTA ends with a copy still on its way to its shared
memory, the status says NVFP4_ERR_TIMEOUT and the next call is right."""
import pytest
import torch

from nvfp4_post_weight_b200 import binding as B
from nvfp4_post_weight_b200.decoder import DecoderLayerSolver, MoELayerSolver
from nvfp4_post_weight_b200.layer import LayerSolver
from test_gpu_gemv import BF16, DEV, F32, acts, by_expert, close, fp4, gated_fp4, sums_fp4, weights

pytestmark = pytest.mark.gpu
TIMEOUT = 6   # NVFP4_ERR_TIMEOUT (a copy in flight at a CTA's end: 9)


class no_waiting:
    def __enter__(self):
        torch.cuda.synchronize()
        B.nvfp4_set_wait_limit_ns(1)

    def __exit__(self, *a):
        torch.cuda.synchronize()
        B.nvfp4_set_wait_limit_ns(0)


# stages a CTA and slots of its ring: 4 of 6, many, as many in each of two CTAs,
# of a pair of matrices, and of experts
CALLS = [("gemv", 5, 20003, 1024), ("gemv", 9, 6144, 8192), ("gemv", 5, 5201, 12544),
         ("swiglu", 3, 20011, 512), ("experts", 40, 2048, 1024)]


@pytest.mark.parametrize("op,n,d_out,d_in", CALLS)
@pytest.mark.parametrize("debug", [False, True])
def test_no_copy_outlives_its_cta(monkeypatch, op, n, d_out, d_in, debug):
    """The debug build looks at every copy's barrier before a CTA ends, and
    records NVFP4_ERR_BOUNDS over the timeout for one that has not landed."""
    E = 40 if op == "experts" else 0
    pair = op == "swiglu"
    assert fp4(n, d_out, d_in, E, pair)
    w = [weights((E, d_out, d_in) if E else (d_out, d_in), s) for s in ((1, 2) if pair else (1,))]
    x = acts(n, d_in, BF16, 3) * 0.1
    y = torch.zeros((n, d_out), dtype=F32, device=DEV)
    offsets = torch.arange(41, dtype=torch.int32, device=DEV)
    ws = B.workspace(B.nvfp4_gemv_workspace_size(n, d_out, d_in, E, pair), DEV)

    def call():
        if op == "gemv":
            B.nvfp4_gemv(x, *w[0], y, ws)
        elif pair:
            B.nvfp4_gemv_swiglu(x, *w, y, ws)
        else:
            B.nvfp4_gemv_experts(x, offsets, *w[0], y, None, ws)

    if debug:
        monkeypatch.setattr(B, "_lib", B.debug_lib())
    for _ in range(5):
        with no_waiting():
            call()
        assert B.nvfp4_workspace_status(ws) == TIMEOUT
    call()
    assert B.nvfp4_workspace_status(ws) == 0
    if E:
        by_expert(lambda r, m: close(y[r], *sums_fp4(x[r], m)), offsets, w[0])
    else:
        close(y, *(gated_fp4 if pair else sums_fp4)(x, *w))


def test_the_solvers_tell_of_a_timed_out_product():
    """Their products take workspaces that go with the call; the word that
    product_status reads stays."""
    layer = LayerSolver(40003, 512, DEV)
    dec = DecoderLayerSolver((("x", {"gate": (20011, 512), "up": (20011, 512)}),), DEV)
    moe = MoELayerSolver(8, 2560, 2048, DEV)
    for codes, scales, sg in ((layer.codes, layer.scales, layer.s_g), dec.weight("gate"),
                              dec.weight("up"), *moe.stacked.values()):
        c, s, g = weights((*sg.shape[:codes.dim() - 2], codes.shape[-2], 2 * codes.shape[-1]), 5)
        codes.copy_(c), scales.copy_(s), sg.copy_(g)
    x = acts(5, 512, BF16, 3) * 0.1
    xm = acts(5, 2560, BF16, 4) * 0.1
    ids = torch.arange(10, dtype=torch.int32, device=DEV).view(5, 2) % 8
    w = torch.rand((5, 2), device=DEV)
    assert fp4(5, 40003, 512) and fp4(5, 20011, 512, 0, True) and fp4(10, 2048, 2560, 8, True)
    calls = ((layer, lambda: layer.linear(x)), (dec, lambda: dec.gated("gate", "up", x)),
             (moe, lambda: moe.forward(xm, ids, w)))
    B.nvfp4_product_status()   # (what other tests timed out)
    for s, call in calls:
        good = call()
        assert s.product_status() == 0
        with no_waiting():
            call()
        assert s.product_status() == TIMEOUT
        assert s.product_status() == 0          # read and cleared
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = call()
        assert s.product_status(side) == 0 and torch.equal(good, again)
