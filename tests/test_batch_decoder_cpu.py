"""What BatchDecoder refuses before it makes anything on a device."""
import types

import numpy as np
import pytest

from int4_gathered_expert_gb300 import synth

torch = pytest.importorskip("torch")

A = synth.AttnShape(Hq=4, Hkv=2, D=64, block_tokens=64)


def make(max_blocks=4, **kw):
    from int4_gathered_expert_gb300.model import BatchDecoder
    cache = types.SimpleNamespace(descs=[], B=1, max_blocks=max_blocks, block_tokens=64)
    return BatchDecoder(types.SimpleNamespace(L=0, H=64), [], A, cache, 1, device="meta", **kw)


@pytest.mark.filterwarnings("ignore::RuntimeWarning")
@pytest.mark.parametrize("cap", [-1.0, float("nan"), float("inf"), 1e39, 1e-46])
def test_caps_that_fp32_does_not_hold(cap):
    """A cap that fp32 holds as 0 would be none at all, one that it holds as infinity an error of every step."""
    with pytest.raises(ValueError, match="cap"):
        make(cap=cap)


def test_a_prefix_and_a_sequence_with_too_many_positions():
    """Each of them fits, both together have more positions than attention takes."""
    with pytest.raises(ValueError, match="positions"):
        make(max_blocks=(1 << 30) // 64, prefix=True)
