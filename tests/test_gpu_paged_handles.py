"""PagedKVCache and PagedBatch as objects that a program keeps: tensors replaced,
changed in place, copied and stored."""
import copy
import gc
import io
import pickle
import weakref

import numpy as np
import pytest
import torch

from gpu_util import to_dev
from test_gpu_paged import World, bits
from w4a16_dequant_gemv_amd import W4A16Error, kv

pytestmark = pytest.mark.gpu

TENSORS = ("k", "v", "k_scale", "v_scale", "k_tail", "v_tail")


def used():
    """A cache of two sequences that has appended and attended, a query and its batch."""
    w = World(2, 2, 64, 64, seed=12)
    w.append([150, 90])
    q = to_dev(w.values(2, 4))
    b = w.batch([1, 1], ctx=[149, 89])
    return w.cache, q, b, w.cache.attend(q, b)


@pytest.mark.parametrize("name", TENSORS)
def test_a_replaced_tensor_is_let_go(name):
    """A program that replaces a pool has the old one's memory back before the next call."""
    c, q, b, want = used()
    old = getattr(c, name)
    gone = weakref.ref(old)
    setattr(c, name, old.clone())
    del old
    gc.collect()
    assert gone() is None
    assert np.array_equal(bits(c.attend(q, b)), bits(want))
    setattr(c, name, getattr(c, name).double())
    with pytest.raises(W4A16Error, match=name):
        c.attend(q, b)


def test_changed_sizes_are_checked():
    c, q, b, want = used()
    c.page = 128
    with pytest.raises(W4A16Error):
        c.attend(q, b)
    c.page = 64
    assert np.array_equal(bits(c.attend(q, b)), bits(want))


@pytest.mark.parametrize("name", TENSORS)
def test_a_tensor_made_smaller_in_place_is_refused(name):
    c, q, b, want = used()
    t = getattr(c, name)
    shape = t.shape
    t.resize_(shape[0] - 1, *shape[1:])                  # its memory stays where it is
    with pytest.raises(W4A16Error):
        c.attend(q, b)
    t.resize_(shape)
    assert np.array_equal(bits(c.attend(q, b)), bits(want))


def test_a_pool_made_smaller_in_place_is_used_as_such():
    """All of its tensors: the pages that are gone are not visible any more."""
    w = World(1, 1, 64, 64, seed=1)
    w.append([200])
    at = int(w.table[0, 1])
    for name in ("k", "v", "k_scale", "v_scale"):
        t = getattr(w.cache, name)
        t.resize_(at, *t.shape[1:])
    hidden = [p for p in range(3) if w.table[0, p] >= at]
    w.attend([1], 4, hidden=hidden)


def test_a_block_table_of_another_shape_in_place():
    """The same number of entries in another shape, and a table turned in place."""
    c, q, b, want = used()
    table = b.block_table
    rows, cols = table.shape
    table.resize_(rows * cols // 2, 2)
    with pytest.raises(W4A16Error):
        c.attend(q, b)
    table.resize_(rows, cols)
    assert np.array_equal(bits(c.attend(q, b)), bits(want))
    square = torch.full((2, 2), -1, dtype=torch.int32, device="cuda")
    batch = kv.PagedBatch(b.cu_q, b.ctx_lens, square, b.slots)
    square.t_()
    with pytest.raises(W4A16Error, match="contiguous"):
        c.attend(q, batch)


@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle", "save"])
def test_copies_of_a_used_cache(how):
    """Copied or stored after calls, as before them; a deep copy goes its own way."""
    c, q, b, want = used()
    if how == "save":
        f = io.BytesIO()
        torch.save((c, b), f)
        f.seek(0)
        c2, b2 = torch.load(f, weights_only=False)
    elif how == "pickle":
        c2, b2 = pickle.loads(pickle.dumps((c, b)))
    else:
        c2, b2 = getattr(copy, how)(c), getattr(copy, how)(b)
    assert np.array_equal(bits(c2.attend(q, b2)), bits(want))
    if how != "copy":
        c2.k_tail.zero_()
        b2.ctx_lens.fill_(1)
        assert not np.array_equal(bits(c2.attend(q, b2)), bits(want))
    assert np.array_equal(bits(c.attend(q, b)), bits(want))
