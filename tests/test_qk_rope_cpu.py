"""What QkRope refuses, before anything is launched."""
import types

import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture()
def QkRope(monkeypatch):
    from int4_gathered_expert_gb300 import model
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: None)
    monkeypatch.setattr(model.L, "e0_qk_rope", lambda *a, **k: pytest.fail("launched"))
    return model.QkRope


SHAPE = types.SimpleNamespace(Hq=4, Hkv=2, D=64)
FREQ = np.ones(32, np.float32)


@pytest.mark.parametrize("axis", [np.full(32, -1), np.r_[np.zeros(31, int), -3], np.full(32, 0.5), np.zeros(31, int), np.full(32, 2)])
def test_axes_that_are_none(QkRope, axis):
    with pytest.raises(ValueError):
        QkRope(SHAPE, FREQ, axis=axis, n_axes=2, device="cpu")


def test_host_tensors(QkRope):
    rope = QkRope(SHAPE, FREQ, device="cpu")
    with pytest.raises(ValueError):
        rope(0, torch.zeros((3, 512), dtype=torch.float16), torch.zeros(3, dtype=torch.int32))


@pytest.mark.parametrize("axes,shape", [(1, (4,)), (1, (3, 1)), (2, (3,)), (2, (6,)), (2, (3, 2)), (2, (1, 6)), (2, ()), (3, (3, 3, 1))])
def test_positions_of_another_shape(QkRope, monkeypatch, axes, shape):
    """[axes, T], or [T] where there is one: not as many numbers in another order."""
    rope = QkRope(SHAPE, FREQ, axis=np.zeros(32, int), n_axes=axes, device="cpu")
    with pytest.raises(ValueError, match="positions are"):
        rope(0, torch.zeros((3, 512), dtype=torch.float16), torch.zeros(shape, dtype=torch.int32))


def test_tables_and_rows_on_devices_of_their_own(QkRope):
    rope = QkRope(SHAPE, FREQ, device="cpu")
    for qkv, pos in (("meta", "cpu"), ("meta", "meta"), ("cpu", "meta")):
        with pytest.raises(ValueError, match="device"):
            rope(0, torch.zeros((3, 512), dtype=torch.float16, device=qkv), torch.zeros(3, dtype=torch.int32, device=pos))
