"""A feed-forward call that fails on the host has enqueued nothing.  The failure is
made on the host: a test hook answers in the CUDA runtime's place."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

ERR_CUDA = 5


@pytest.fixture
def refused():
    import async_copy_pipelined_gb300 as pg
    lib = pg.lib()
    lib.gemm_testing_refuse_smem_limit(1)
    try:
        yield
    finally:
        lib.gemm_testing_refuse_smem_limit(0)


def _bf16(*shape):
    import torch
    return torch.randn(shape, device="cuda").bfloat16()


@pytest.mark.parametrize("rows", [4, 300])
def test_a_gradient_that_fails_has_not_touched_its_workspace(rows, refused):
    import torch
    import async_copy_pipelined_gb300 as pg
    lib = pg.lib()
    width, hidden = 64, 136
    dh, gate, up = (_bf16(rows, hidden) for _ in range(3))
    x, wg, wu = _bf16(rows, width), _bf16(width, hidden), _bf16(width, hidden)
    results = [torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda")
               for s in ((rows, width), (width, hidden), (width, hidden))]
    need = ctypes.c_size_t()
    assert lib.gated_projection_backward_workspace(rows, width, hidden, ctypes.byref(need)) == 0
    ws = torch.full((need.value,), 77, dtype=torch.uint8, device="cuda")
    st = lib.gated_projection_backward(
        rows, width, hidden, dh.data_ptr(), hidden, x.data_ptr(), width, wg.data_ptr(), hidden, wu.data_ptr(), hidden,
        gate.data_ptr(), hidden, up.data_ptr(), hidden, results[0].data_ptr(), width, results[1].data_ptr(), hidden,
        results[2].data_ptr(), hidden, 0, ws.data_ptr(), need.value, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == ERR_CUDA
    assert (ws == 77).all() and all((t == 7.0).all() for t in results)


def test_calls_that_fail_raise_and_the_next_ones_are_right():
    import torch
    import async_copy_pipelined_gb300 as pg
    x, wg, wu, wd = _bf16(300, 64), _bf16(64, 136), _bf16(64, 136), _bf16(136, 64)

    def step():
        h, gate, up = pg.gated_projection(x, wg, wu, save=True)
        q, s = pg.quantize_fp8(h)
        d, t = pg.quantize_fp8(wd, "block")
        return (h, pg.gemm_fp8(q, d, s, t), *pg.gated_projection_backward(h, x, wg, wu, gate, up))

    want = step()
    h, gate, up = pg.gated_projection(x, wg, wu, save=True)
    q, s = pg.quantize_fp8(h)
    d, t = pg.quantize_fp8(wd, "block")
    calls = (lambda: pg.gated_projection(x, wg, wu), lambda: pg.gated_projection(x[:2], wg, wu),
             lambda: pg.gated_projection_backward(h, x, wg, wu, gate, up), lambda: pg.gemm_fp8(q, d, s, t),
             lambda: pg.gemm_fp8(q[:2], d, s[:2], t))
    try:
        pg.lib().gemm_testing_refuse_smem_limit(1)
        for call in calls:
            with pytest.raises(pg.GemmError) as e:
                call()
            assert e.value.status == ERR_CUDA
    finally:
        pg.lib().gemm_testing_refuse_smem_limit(0)
    assert all(torch.equal(a, b) for a, b in zip(step(), want))
    assert pg.device_status()[0] == 0
