"""Refusals of the linear layers in 8-bit floating point, without a GPU: every case fails a host
check, so the pointers are never dereferenced and nothing is launched."""
import pytest
import torch

E_ARG, E_ALIGN, E_UNSUPPORTED, E_WORKSPACE = -1, -2, -3, -4
P = 0x1000


def _lib():
    import __graft_entry__
    __graft_entry__.build()
    from block_diffusion_speculative_02_gb300 import dflash
    return dflash, dflash.load_library()


def test_norm_rows_refuses():
    _, lib = _lib()

    def f(rows=4, cols=256, x=P, xp=256, r=None, rp=0, w=None, eps=1e-6, s=None, sp=0, q=P,
          scale=P):
        return lib.dflash_fp8_norm_rows(rows, cols, x, xp, r, rp, w, eps, s, sp, q, scale, None)

    assert f(rows=-1) == f(cols=0) == f(x=None) == f(q=None) == f(scale=None) == E_ARG
    assert f(eps=-1.0) == f(eps=float("nan")) == f(eps=float("inf")) == E_ARG
    assert f(xp=255) == f(xp=-256) == f(r=P, rp=0) == f(s=P, sp=248) == E_ARG
    assert f(cols=250) == f(cols=8) == f(cols=32784, xp=32784) == E_UNSUPPORTED
    assert f(xp=260) == f(x=P + 2) == f(r=P + 8, rp=256) == f(w=P + 2) == E_ALIGN
    assert f(s=P + 4, sp=256) == f(q=P + 1) == f(scale=P + 2) == E_ALIGN
    assert f(rows=0, x=None, q=None, scale=None) == 0                 # nothing to do
    # sum_out in the place of x or of the residual, its rows elsewhere
    assert f(s=P, sp=264) == f(x=2 * P, r=P, rp=256, s=P, sp=512) == E_ARG


def test_silu_mul_refuses():
    _, lib = _lib()

    def f(rows=4, cols=256, x=P, xp=512, q=P, scale=P):
        return lib.dflash_fp8_silu_mul(rows, cols, x, xp, q, scale, None)

    assert f(rows=-1) == f(cols=0) == f(x=None) == f(q=None) == f(scale=None) == E_ARG
    assert f(xp=504) == E_ARG
    assert f(cols=24) == E_UNSUPPORTED
    assert f(xp=516) == f(x=P + 2) == f(q=P + 8) == f(scale=P + 1) == E_ALIGN
    assert f(rows=2 ** 31 - 1, cols=2 ** 31 - 16, xp=2 ** 33) == E_UNSUPPORTED   # too many blocks
    assert f(rows=0, x=None) == 0


def test_weight_refuses():
    _, lib = _lib()

    def f(g=1, n=64, k=256, w=P, q=P, scale=P):
        return lib.dflash_fp8_weight(g, n, k, w, q, scale, None)

    assert f(g=0) == f(n=0) == f(k=0) == f(w=None) == f(q=None) == f(scale=None) == E_ARG
    assert f(k=40) == f(g=2 ** 20, n=2 ** 20, k=2 ** 20) == E_UNSUPPORTED
    assert f(w=P + 2) == f(q=P + 4) == f(scale=P + 2) == E_ALIGN


def test_products_refuse():
    _, lib = _lib()

    def linear(m=4, n=64, k=256, x=P, xs=P, w=P, ws=P, out=P, pitch=64, wsp=P, nws=256):
        return lib.dflash_fp8_linear(m, n, k, x, xs, w, ws, out, pitch, wsp, nws, None)

    def grouped(m=4, src=4, g=3, n=64, k=256, x=P, xs=P, w=P, ws=P, start=P, rows=None, out=P,
                pitch=64, wsp=P, nws=256):
        return lib.dflash_fp8_grouped(m, src, g, n, k, x, xs, w, ws, start, rows, out, pitch, wsp,
                                      nws, None)

    for f in (linear, grouped):
        assert f(m=-1) == f(n=0) == f(k=0) == f(pitch=63) == E_ARG
        assert f(x=None) == f(xs=None) == f(w=None) == f(ws=None) == f(out=None) == E_ARG
        assert f(k=264) == E_UNSUPPORTED
        assert f(m=2 ** 31 - 1, pitch=64) == f(n=2 ** 31 - 1, pitch=2 ** 31) == E_UNSUPPORTED
        assert f(x=P + 8) == f(w=P + 8) == f(xs=P + 2) == f(ws=P + 2) == f(out=P + 1) == E_ALIGN
        assert f(wsp=None) == f(nws=63) == E_WORKSPACE
        assert f(wsp=P + 2) == E_ALIGN
        assert f(m=0, x=None, out=None) == 0
    assert grouped(g=0) == grouped(src=-1) == grouped(start=None) == E_ARG
    assert grouped(src=5) == E_ARG                                    # which rows of x?
    assert grouped(src=0, rows=P) == E_ARG
    assert grouped(g=1025) == grouped(g=1024, n=2 ** 22, pitch=2 ** 22) == E_UNSUPPORTED


def test_failure_injection_reaches_every_call(monkeypatch):
    _, lib = _lib()
    calls = {"dflash_fp8_norm_rows": (0, 0, None, 0, None, 0, None, 0.0, None, 0, None, None, None),
             "dflash_fp8_silu_mul": (0, 0, None, 0, None, None, None),
             "dflash_fp8_weight": (0, 0, 0, None, None, None, None),
             "dflash_fp8_linear": (0,) * 3 + (None,) * 5 + (0, None, 0, None),
             "dflash_fp8_grouped": (0,) * 5 + (None,) * 7 + (0, None, 0, None)}
    for name, args in calls.items():
        monkeypatch.setenv("DFLASH_FAULT_INJECT", name)
        assert getattr(lib, name)(*args) == -5, name
        monkeypatch.setenv("DFLASH_FAULT_INJECT", name + ":-4")
        assert getattr(lib, name)(*args) == -4, name


def test_binding_names_what_is_wrong():
    """(CPU tensors are on "device" -1.)"""
    d, _ = _lib()
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    assert d._matrix(x, -1, "x", (4, 32)) == (x.data_ptr(), 32)
    assert d._matrix(x[:, :16], -1, "x", (4, 16)) == (x.data_ptr(), 32)
    assert d._matrix(x[1:2, :16], -1, "x", (1, 16))[1] == 16          # one row has no pitch
    for bad, shape in ((x.float(), (4, 32)), (x[:, ::2], (4, 16)), (x, (4, 16)), (None, (4, 32)),
                       ("x", (4, 32))):
        with pytest.raises(ValueError, match="^x"):
            d._matrix(bad, -1, "x", shape)
    q = torch.zeros(4, 32, dtype=torch.uint8).view(d.F8)
    assert d._whole(q, -1, d.F8, (4, 32), "q") == q.data_ptr()
    for bad in (q[:, :16], q.view(torch.uint8), q.view(8, 16), None, q[0]):
        with pytest.raises(ValueError, match="^q"):
            d._whole(bad, -1, d.F8, (4, 32), "q")
    for bad in (None, q[0], 3):
        with pytest.raises(ValueError, match="dimensions"):
            d._shape(bad, 2, "q")
    a, b = d.alloc_fp8_rows(5, 200, device="cpu")
    assert a.shape == (5, 200) and b.shape == (2, 5) and a.dtype is d.F8
    a, b = d.alloc_fp8_weight(3, 130, 144, device="cpu")
    assert a.shape == (3, 130, 144) and b.shape == (3, 2, 2)
