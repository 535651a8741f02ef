"""What the Python binding of linear attention and rotary positions makes of its arguments,
without a GPU: descriptors hold the values of their own call."""
import pytest

import test_sequence_layer_amd as ttt

torch = pytest.importorskip("torch")


def _desc(scale, B=1, H=2, T=5, d=16):
    q = torch.zeros(B, H, T, d)
    return ttt._attn_desc(q, q, q, torch.zeros(H), None, None, scale, torch.zeros(B, H, T, d))[0]


@pytest.mark.parametrize("make", [lambda x: torch.tensor(x), lambda x: torch.nn.Parameter(torch.tensor(x))])
def test_scale_is_read_at_every_call(make):
    """A scale kept in a tensor and changed in place: the next descriptor holds the new value."""
    scale = make(0.5)
    assert _desc(scale).scale == 0.5
    with torch.no_grad():
        scale.mul_(4)
    assert _desc(scale).scale == 2.0
    assert _desc(2.0).scale == 2.0 and _desc(torch.tensor(-1.0)).scale == -1.0


def test_cached_descriptors_keep_no_tensor():
    _desc(torch.tensor(0.25))
    flat = lambda x: [z for y in x for z in flat(y)] if isinstance(x, tuple) else [x]  # noqa: E731
    assert not any(torch.is_tensor(x) for key in ttt._attn_descs for x in flat(tuple(key)))
