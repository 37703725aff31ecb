"""Shared-memory limits of the routing and product kernels: sizes at the edge of
what needs no setting, and calls of different sizes from several threads at once
(the limit is state of a kernel that they share)."""
import subprocess
import sys
import threading
import os

import pytest
import torch

from nvfp4_post_weight_b200 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SORT = """
import sys, torch
from nvfp4_post_weight_b200 import binding as B
E, T, k = int(sys.argv[1]), int(sys.argv[2]), 2
i32 = dict(dtype=torch.int32, device="cuda:0")
ids = torch.arange(T * k, **i32).view(T, k) % E
off, rows, pos = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty((T, k), **i32)
B.nvfp4_moe_sort(ids, off, rows, pos)
order = torch.argsort(ids.flatten(), stable=True)
assert torch.equal(rows.long(), order // k) and off[-1] == T * k
"""


@pytest.mark.parametrize("E", [248, 249, 371, 372, 373])
@pytest.mark.parametrize("T", [400, 4000])
def test_sort_of_experts_at_the_edge_of_the_default_limit(E, T):
    """33 ints an expert and the static shared memory beside them: the first sort
    of a process, before any larger one has raised the limit."""
    subprocess.run([sys.executable, "-c", SORT, str(E), str(T)], check=True, cwd=ROOT, timeout=300)


def together(*calls, times=3000):
    """Runs the calls over and over in a thread each; the statuses but NVFP4_OK."""
    bad = []

    def loop(call):
        for _ in range(times):
            status = call()
            if status:
                bad.append(status)

    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return bad


def test_sorts_of_several_threads():
    L = B.lib()
    ids = torch.zeros((64, 2), dtype=torch.int32, device=DEV)

    def sorts(E):
        off, rows, pos = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (E + 1, 128, 128))
        ptrs = [t.data_ptr() for t in (off, rows, pos)]
        st = torch.cuda.Stream()
        keep = (off, rows, pos, st)
        return lambda: keep and L.nvfp4_moe_sort(ids.data_ptr(), 4, 64, 2, E, *ptrs, st.cuda_stream)

    assert together(*[sorts(E) for E in (1024, 400, 800, 380)]) == []


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_products_of_several_threads(dtype):
    """Sizes that one kernel serves with 60 to 80 KB of shared memory of bf16 tokens,
    84 to 112 KB of fp32 ones."""
    L = B.lib()
    d_out, d_in = 16, 16384 if dtype == torch.bfloat16 else 512
    codes = torch.randint(0, 256, (d_out, d_in // 2), dtype=torch.uint8, device=DEV)
    scales = torch.full((d_out, d_in // 16), 56, dtype=torch.uint8, device=DEV)
    sg = torch.ones(1, device=DEV)
    w = [t.data_ptr() for t in (codes, scales, sg)]

    def products(n):
        assert B.nvfp4_gemv_workspace_size(n, d_out, d_in, dtype=dtype) == 0
        x, y = torch.ones((n, d_in), dtype=dtype, device=DEV), torch.empty((n, d_out), device=DEV)
        st = torch.cuda.Stream()
        keep = (x, y, st, codes, scales, sg)
        t = 0 if dtype == torch.bfloat16 else 1
        return lambda: keep and L.nvfp4_gemv(x.data_ptr(), t, n, *w, d_out, d_in, y.data_ptr(), 1,
                                             None, 0, st.cuda_stream)

    assert together(*[products(n) for n in (32, 24, 30, 25)], times=10000) == []


def test_phases_of_products_and_routing():
    """The profile's phases, by the public header's numbers."""
    import ctypes
    import re
    src = open(os.path.join(ROOT, "include", "nvfp4pw.h")).read()
    phase = {m[0]: int(m[1]) for m in re.findall(r"NVFP4_(\w+) = (\d+)", src)}
    n = phase["NUM_PHASES"]
    ms, launches = (ctypes.c_double * n)(), (ctypes.c_longlong * n)()
    i32 = dict(dtype=torch.int32, device=DEV)
    ids, off, rows, pos = (torch.zeros(s, **i32) for s in ((4, 2), (4,), (8,), (4, 2)))
    x, y = torch.ones((4, 32), device=DEV), torch.empty((4, 16), device=DEV)
    w = (torch.zeros((16, 16), dtype=torch.uint8, device=DEV),
         torch.zeros((16, 2), dtype=torch.uint8, device=DEV), torch.ones(1, device=DEV))
    assert B.lib().nvfp4_profile_begin() == 0
    B.nvfp4_gemv(x, *w, y)
    B.nvfp4_moe_sort(ids, off, rows, pos)
    B.nvfp4_moe_gather(x, pos, torch.empty((8, 32), device=DEV))
    assert B.lib().nvfp4_profile_end(ms, launches, n) == 0
    assert launches[phase["PHASE_PRODUCT"]] == 1 and launches[phase["PHASE_ROUTE"]] == 2
    assert ms[phase["PHASE_PRODUCT"]] > 0 and ms[phase["PHASE_ROUTE"]] > 0
