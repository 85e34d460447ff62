"""Which kernel a product goes to, on the host."""
import pytest


def _dfl():
    import __graft_entry__
    __graft_entry__.build()
    import block_diffusion_speculative_02_gb300 as dfl
    return dfl


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
