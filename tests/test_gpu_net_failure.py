"""Failure detection of the weight gradient without a GPU fault: its bounded waits run
out on purpose (exponents that never come), the kernel waits for its copies under way,
flags the error and returns, the host reads GS_ERR_TIMEOUT, and the next call on the
same workspace is right."""
import ctypes as C

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


@pytest.mark.parametrize("T,N,K,stops", [
    (100, 40, 64, (0,)),                # two steps, one cluster
    (20000, 512, 512, (0, 8, 16)),      # 17 steps a cluster: first batch, rings full, one left
    (3000, 2600, 2050, (0, 8, 24)),     # whole tiles first: several runs of products
])
def test_wgrad_waits_run_out_and_context_survives(gs, T, N, K, stops):
    L = gs.lib()
    vp = C.c_void_p
    L.gs_selftest_wgrad_timeout.restype = C.c_int
    L.gs_selftest_wgrad_timeout.argtypes = [C.c_int64, C.c_int32, C.c_int32, vp, vp, vp, vp, vp, C.c_size_t,
                                            C.c_int32, vp]
    g = torch.Generator(device="cuda").manual_seed(T)
    dy = torch.randn(T, N, generator=g, device="cuda").bfloat16()
    q, e = gs.act8_empty(T, K)
    gs.gs_act8_encode(torch.randn(T, K, generator=g, device="cuda"), q, e)
    ws = torch.zeros(gs.gs_act8_wgrad_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    want, got = (torch.empty(N, K, device="cuda") for _ in range(2))
    gs.gs_act8_wgrad(dy, q, e, want, ws)
    stream = torch.cuda.current_stream().cuda_stream
    for steps in stops:
        st = L.gs_selftest_wgrad_timeout(T, N, K, dy.data_ptr(), q.data_ptr(), e.data_ptr(), got.data_ptr(),
                                         ws.data_ptr(), ws.numel(), steps, stream)
        assert st == gs.GS_ERR_TIMEOUT, steps
        assert gs.gs_workspace_status(ws) == gs.GS_OK  # read and cleared
        got.fill_(7.0)
        gs.gs_act8_wgrad(dy, q, e, got, ws)
        assert gs.gs_workspace_status(ws) == gs.GS_OK and torch.equal(got, want), steps
    # exponents enough for every step: the same kernel ends as usual
    st = L.gs_selftest_wgrad_timeout(T, N, K, dy.data_ptr(), q.data_ptr(), e.data_ptr(), got.data_ptr(),
                                     ws.data_ptr(), ws.numel(), 1 << 20, stream)
    assert st == gs.GS_OK and torch.equal(got, want)
