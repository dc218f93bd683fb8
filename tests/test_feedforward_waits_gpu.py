"""Waits of the 8-bit product's pair kernel for its scales: one that runs out ends
the call and is recorded, whichever K block it is of.  Nothing is faulted: the
scales of one block are simply never announced."""
import pytest

FAMILY_FP8 = 10
PRODUCER, MMA, EPILOGUE = 2, 3, 4


def test_the_hook_refuses_what_is_no_position():
    import async_copy_pipelined_gb300 as pg
    pg.build()
    assert pg.lib().gemm_testing_withhold_scales(-2) == 1
    assert pg.lib().gemm_testing_withhold_scales(-1) == 0


def _operands(M, N, K, b_group):
    import torch
    import async_copy_pipelined_gb300 as pg
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, sa = pg.quantize_fp8(torch.randn((K, M), generator=g, device="cuda"), "column")  # transposed: pairs of CTAs
    b, sb = pg.quantize_fp8(torch.randn((K, N), generator=g, device="cuda"), b_group)
    return a.t(), b, sa.t(), sb


# (M, N, K), K blocks of a CTA with most of them: a tile a pair; several tiles in
# turn; two and four pairs to a tile's contraction.
CASES = [((2048, 2048, 512), 4), ((4096, 4096, 512), 16), ((1500, 1500, 4096), 16), ((400, 400, 4096), 8),
         ((256, 256, 100), 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("b_group", ["block", "column"])
@pytest.mark.parametrize("size,blocks", CASES)
def test_scales_that_never_come_are_reported(size, blocks, b_group):
    """The last blocks of a CTA are those where no other warp would notice: the
    tensor core needs no further accumulator."""
    import torch
    import async_copy_pipelined_gb300 as pg
    operands = _operands(*size, b_group)
    lib = pg.lib()
    for dtype in (torch.float32, torch.bfloat16):
        want = pg.gemm_fp8(*operands, dtype=dtype)
        assert pg.device_status()[0] == 0
        for position in sorted({0, 1, blocks // 2, blocks - 2, blocks - 1}):
            if not 0 <= position < blocks:
                continue
            try:
                pg.testing_set_hooks(10_000_000, -1)
                assert lib.gemm_testing_withhold_scales(position) == 0
                pg.gemm_fp8(*operands, dtype=dtype)
                st, detail = pg.device_status()
            finally:
                pg.testing_set_hooks(0, -1)
                lib.gemm_testing_withhold_scales(-1)
            assert st == 6 and detail & 0xFF == FAMILY_FP8, (position, st, detail)
            assert (detail >> 8) & 0xFF in (PRODUCER, MMA, EPILOGUE), (position, detail)
            if position == blocks - 1:
                assert (detail >> 8) & 0xFF == EPILOGUE
            assert torch.equal(pg.gemm_fp8(*operands, dtype=dtype), want)
            assert pg.device_status()[0] == 0


@pytest.mark.gpu
def test_a_position_that_no_cta_reaches_withholds_nothing():
    import torch
    import async_copy_pipelined_gb300 as pg
    operands = _operands(2048, 2048, 512, "block")
    want = pg.gemm_fp8(*operands)
    try:
        pg.lib().gemm_testing_withhold_scales(4)
        assert torch.equal(pg.gemm_fp8(*operands), want)
    finally:
        pg.lib().gemm_testing_withhold_scales(-1)
    assert pg.device_status()[0] == 0
