"""The binding of the calls over a 4-bit cache on the host: what a view keeps between calls, and
what it refuses.  (CPU tensors are on "device" -1.)"""
import copy
import pickle
import weakref

import pytest
import torch

HOST = -1


def _dflash():
    from block_diffusion_speculative_02_gb300 import dflash
    return dflash


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _view4(pages=9, batch=2, hkv=2, d=64):
    dflash = _dflash()
    return dflash.KV4View(dflash.alloc_kv4_cells(pages, hkv, 16, d, device="cpu"), _i32(batch), 64,
                          _i32(batch, 4), _i32(pages), _i32(1), 16, _i32(hkv), _i32(hkv))


def _view16(pages=9, batch=2):
    dflash = _dflash()
    return dflash.KVView(None, None, _i32(batch), 64, _i32(batch, 4), _i32(pages), _i32(1), 16)


def _use(view):
    """What a call over the cells, or the page reservation, makes of a view."""
    dflash = _dflash()
    if isinstance(view, dflash.KV4View):
        dflash._view_struct(view, HOST, 2, 0, 0)
        return dflash._view_struct(view, HOST, 2, 2, 64)
    return dflash._view_struct(view, HOST, 2, 0, 0)


@pytest.mark.parametrize("make", [_view4, _view16])
@pytest.mark.parametrize("clone", [copy.deepcopy, copy.copy,
                                   lambda v: pickle.loads(pickle.dumps(v))])
def test_used_views_copy_and_pickle(make, clone):
    view = make()
    _use(view)
    other = clone(view)
    assert type(other) is type(view) and other.capacity == view.capacity
    assert torch.equal(other.page_table, view.page_table)
    c = _use(other)
    pages = c.kv if hasattr(c, "kv") else c
    assert pages.page_table == other.page_table.data_ptr()
    assert pages.seq_len == other.seq_len.data_ptr()


@pytest.mark.parametrize("field", ["cells", "page_table", "free_list", "k_exp"])
def test_exchanged_tensors_are_let_go(field):
    """A tensor that leaves a view is freed then, not at the view's next call."""
    view = _view4()
    _use(view)
    old = weakref.ref(getattr(view, field))
    setattr(view, field, getattr(view, field).clone())
    assert old() is None
    c = _use(view)
    here = {"cells": c.kv.k, "page_table": c.kv.page_table, "free_list": c.kv.free_list,
            "k_exp": c.k_exp}
    assert here[field] == getattr(view, field).data_ptr()
    old = weakref.ref(view.cells)
    view.cells = None
    assert old() is None


def test_page_struct_is_kept_whatever_the_cells_are():
    """The reservation's struct does not depend on the cells: exchanging them leaves it valid."""
    dflash = _dflash()
    view = _view4()
    c = dflash._view_struct(view, HOST, 2, 0, 0)
    view.cells = None
    assert dflash._view_struct(view, HOST, 2, 0, 0) is c


def test_another_tensor_at_the_same_address_is_checked():
    """The kept struct belongs to the tensors it was made of, not to their addresses."""
    view = _view4()
    _use(view)
    view.k_exp = view.k_exp.view(torch.float32)
    with pytest.raises(ValueError):
        _use(view)


def test_a_tensor_turned_in_place_is_refused():
    """A table transposed in place keeps its address and, if square, its shape."""
    view = _view4(batch=4)
    dflash = _dflash()
    use = lambda: dflash._view_struct(view, HOST, 4, 2, 64)  # noqa: E731
    use()
    view.page_table.t_()
    with pytest.raises(ValueError, match="page_table"):
        use()


@pytest.mark.parametrize("field", ["cells", "seq_len", "free_list", "free_count"])
def test_a_view_without_a_tensor_is_a_value_error(field):
    view = _view4()
    setattr(view, field, None)
    with pytest.raises(ValueError, match=field):
        _use(view)


def test_a_missing_or_foreign_argument_is_a_value_error():
    dflash = _dflash()
    for bad in (None, [0, 0], 7):
        with pytest.raises(ValueError, match="start"):
            dflash._on(bad, HOST, torch.int32, 2, "start")
        with pytest.raises(ValueError, match="ws"):
            dflash._ws_on(bad, HOST)
        with pytest.raises(ValueError, match="q must"):
            dflash._rows_on(bad, HOST, 2, 1, 64, "q")
    assert dflash._opt(None, HOST, torch.int32, 2, "k_exp") is None
    view = _view4()
    view.page_table = [[0] * 4] * 2
    with pytest.raises(ValueError, match="page_table"):
        _use(view)


def test_a_single_row_has_any_pitch():
    """The stride of an axis of one row says nothing: slices of one odd row are taken."""
    dflash = _dflash()
    for width in (8 * 64 + 3, 1000):
        rows = torch.zeros(3, width, dtype=torch.bfloat16)
        heads = rows[:, 64:64 + 2 * 64].unflatten(1, (2, 64))[1:2]
        assert heads.stride(0) == width
        assert dflash._rows_on(heads, HOST, 1, 2, 64, "q")[1] % 8 == 0
    two = torch.zeros(2, 515, dtype=torch.bfloat16)[:, :128].unflatten(1, (2, 64))
    assert dflash._rows_on(two, HOST, 2, 2, 64, "q")[1] == 515


def test_a_view_subclass_keeps_its_properties():
    """Setting and deleting fields goes through a subclass's own descriptors."""
    dflash = _dflash()
    seen = []

    class Watched(dflash.KV4View):
        @property
        def note(self):
            return len(seen)

        @note.setter
        def note(self, value):
            seen.append(value)

    view = _view4()
    watched = Watched(*(getattr(view, f) for f in ("cells", "seq_len", "capacity", "page_table",
                                                   "free_list", "free_count", "page_size")))
    watched.note = 5
    assert seen == [5] and watched.note == 1
    _use(watched)
    del watched.k_exp                                   # back to the class's None
    assert watched.k_exp is None and _use(watched).k_exp is None


@pytest.mark.parametrize("cache", [None, "view", _view16])
def test_a_cache_that_is_no_4_bit_view_is_a_value_error(cache):
    dflash = _dflash()
    with pytest.raises(ValueError, match="KV4View"):
        dflash._view_struct(cache() if callable(cache) else cache, HOST, 2, 2, 64)
    if not callable(cache):
        with pytest.raises(ValueError, match="KVView"):
            dflash._view_struct(cache, HOST, 2, 0, 0)
