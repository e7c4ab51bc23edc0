"""Objects that hold tensors let go of them with their last reference, without
the cycle collector (which does not know how much GPU memory waits for it)."""
from __future__ import annotations

import gc
import weakref

import pytest

torch = pytest.importorskip("torch")
ar = pytest.importorskip("reduce_scatter_amd", reason="libar.so not built")


@pytest.fixture(autouse=True)
def no_collector():
    gc.collect()
    gc.disable()
    yield
    gc.enable()


def gradients():
    return [torch.zeros(3), torch.zeros(4, 6).t()]


def gone(build):
    tensors = gradients()
    refs = [weakref.ref(t) for t in tensors]
    keep = build(tensors)
    del tensors
    return keep, lambda: all(r() is None for r in refs)


def test_a_dropped_list_frees_its_tensors():
    lst, freed = gone(ar.GradList)
    assert not freed()
    del lst
    assert freed()


def test_a_list_compared_with_itself_and_others():
    lst, freed = gone(ar.GradList)
    outs, outs_freed = gone(ar.GradList)
    assert lst.like(lst) and lst.like(outs) and lst.like(outs) and outs.like(lst)
    del outs                       # the list remembers whom it was like, and does not keep it
    assert outs_freed() and not freed()
    other = ar.GradList(gradients())
    assert lst.like(other) and not lst.like(ar.GradList([torch.zeros(4)]))
    assert lst.like(other)
    del lst
    assert freed()


def test_shapes_go_with_their_last_reference():
    for build in (lambda: ar.NormShape(4, 16, 2, "f32"), lambda: ar.EmbedShape(4, [8, 8], 16, "f32")):
        shape = build()
        ref = weakref.ref(shape)
        del shape
        assert ref() is None
