"""What the binding hands to the library's layer operators for tensors of unusual
layouts, without a GPU: the library is replaced by a record of its calls, and
host tensors say that they are on a device."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
ar = pytest.importorskip("reduce_scatter_amd", reason="libar.so not built")

from reduce_scatter_amd import _binding as b  # noqa: E402

ADDR = 1 << 24


class OnDevice(torch.Tensor):
    index = 0

    def get_device(self):
        return type(self).index


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def calls(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(b, "_lib", r)
    monkeypatch.setattr(b, "_device", lambda: 0)
    monkeypatch.setattr(OnDevice, "index", 0)
    return r.calls


def tensor(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


def backward(x, rows, width):
    ar.ar_reduce_norm_backward(x, ar.NormShape(rows, width, 1, "f32"), ADDR, ADDR * 2, ADDR * 3, ADDR * 4, stream=0)


@pytest.mark.parametrize("x", [tensor(1, 64).expand(4, 64), tensor(1, 1, 64).expand(2, 2, 64),
                               tensor(64).as_strided((4, 64), (0, 1)), tensor(256).as_strided((4, 64), (63, 1))])
def test_rows_that_share_memory_are_refused(calls, x):
    """A pitch of 0 means the width to the library, which would read past a row that all rows share."""
    with pytest.raises(ValueError, match="pitch"):
        backward(x, 4, 64)
    assert not calls


def test_rows_apart_and_one_row(calls):
    backward(tensor(4, 70)[:, :64], 4, 64)
    backward(tensor(4, 64), 4, 64)
    backward(tensor(64), 1, 64)
    backward(tensor(1, 64).expand(1, 64), 1, 64)
    assert [args[1] for _, args in calls] == [70, 64, 64, 64]


def test_what_was_looked_over_on_another_device_is_looked_over_again(calls, monkeypatch):
    """A list or table that fits the current device does not fit another one that becomes current."""
    grads = ar.GradList([tensor(4), tensor(5)])
    table, em = ar.pointers([tensor(8, 16), tensor(8, 16)]), ar.EmbedShape(4, [8, 8], 16, "f32")
    partials, nm = ar.pointers([tensor(4, 16)]), ar.NormShape(4, 16, 1, "f32")
    todo = [lambda: ar.ar_grad_norm(grads, ADDR, stream=0), lambda: ar.ar_clip_grads(grads, grads, ADDR, 1.0, stream=0),
            lambda: ar.ar_embedding(table, em, ADDR, ADDR * 2, stream=0),
            lambda: ar.ar_embedding_backward(ADDR, em, ADDR * 2, table, stream=0),
            lambda: ar.ar_reduce_norm(partials, nm, ADDR, out=ADDR * 2, stream=0)]
    for f in todo + todo:
        f()
    done = len(calls)
    assert done == 2 * len(todo)
    monkeypatch.setattr(b, "_device", lambda: 1)
    for f in todo:
        with pytest.raises(ValueError, match="current device"):
            f()
    assert len(calls) == done
    monkeypatch.setattr(b, "_device", lambda: 0)
    for f in todo:
        f()
    assert len(calls) == done + len(todo)


def test_rows_of_one_position_and_of_divided_columns(calls):
    """The rows of x as [batch, 1, width], cut from a longer buffer or not, and packed rows whose columns are divided."""
    whole = tensor(4, 7, 64)
    backward(whole[:, 6:], 4, 64)                      # the last position of each sequence
    backward(whole[:, 6:, :48], 4, 48)
    backward(tensor(4, 1, 64), 4, 64)
    backward(tensor(4, 1, 1, 64), 4, 64)
    backward(tensor(2, 1, 2, 64), 4, 64)
    backward(whole[:1, :1], 1, 64)
    backward(tensor(4, 8, 8), 4, 64)
    backward(tensor(4, 1, 70)[..., :64], 4, 64)
    assert [args[1] for _, args in calls] == [448, 448, 64, 64, 64, 64, 64, 70]
    del calls[:]
    # rows that are not at one pitch; divided rows that are not packed
    for x, rows, width in ((whole[:, 5:], 8, 64), (tensor(4, 10, 8)[:, :8], 4, 64), (tensor(2, 4, 64).transpose(0, 1), 8, 64)):
        with pytest.raises(ValueError, match="strides|need more"):
            backward(x, rows, width)
    assert not calls
    backward(whole[:, :, :48], 28, 48)                 # but these are
    assert calls[0][1][1] == 64
