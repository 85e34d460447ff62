"""Which kernel a product goes to, on the host."""
import pytest


def _dfl():
    import __graft_entry__
    __graft_entry__.build()
    import block_diffusion_speculative_02_gb300 as dfl
    return dfl


def test_cases_for_each_kernel_go_to_it():
    """The sizes that the GPU tests name a kernel for reach all of them, on 152 SMs."""
    dfl = _dfl()
    from tests.test_gpu_fp8_kernels import LINEAR, STREAMS, TILES, WHOLE
    for plan, e, m, n, k, index in TILES + STREAMS + WHOLE:
        assert dfl.dflash_fp8_plan(m, n, k, e, index, 152) == plan, (e, m, n, k, index)
    for plan, m, n, k in LINEAR:
        assert dfl.dflash_fp8_plan(m, n, k, num_sms=152) == plan, (m, n, k)
    grouped = {(p[:2], i) for p, _, _, _, _, i in TILES + STREAMS + WHOLE}
    assert grouped == {((r, 128), i) for r in (16, 32, 64) for i in (False, True)} | {
        ((128, 256), True), ((128, 128), False), ((128, 256), False), ((256, 256), False)}
    assert {p[:2] for p, *_ in LINEAR} == {(16, 128), (32, 128), (64, 128), (128, 128), (128, 256),
                                           (256, 256)}
    for i in (False, True):
        assert {(p[0], p[2]) for p, _, _, _, _, j in STREAMS if i == j} >= {
            (16, 2), (16, 8), (32, 8), (64, 4)} if i else {(16, 8), (32, 4), (64, 4)}


def test_plan_refuses():
    dfl = _dfl()
    for bad in ((0, 16, 16), (1, 0, 16), (1, 16, 0), (1, 16, 16, -1), (1, 16, 16, 0, False, -1)):
        with pytest.raises(dfl.DFlashError, match="invalid"):
            dfl.dflash_fp8_plan(*bad)
    for bad in ((1, 16, 24), (1, 16, 16, 1025), (2 ** 31 - 1, 16, 16), (1, 2 ** 22, 16, 1024)):
        with pytest.raises(dfl.DFlashError, match="unsupported"):
            dfl.dflash_fp8_plan(*bad, num_sms=152)
    with pytest.raises(ValueError, match="2\\^31"):
        dfl.dflash_fp8_plan(2 ** 32 + 1, 16, 16, num_sms=152)
