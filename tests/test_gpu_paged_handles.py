"""PagedKVCache and PagedBatch as objects that a program keeps: tensors replaced,
changed in place, copied and stored."""
import gc
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
