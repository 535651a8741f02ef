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


def test_sizes_past_32_bits_are_refused():
    """Expanded tensors of 2^32 + 5 tokens, heads or sequences: not taken for 5."""
    n = (1 << 32) + 5
    x = torch.zeros(1, 1, 1, 16)
    for shape in ((1, 1, n, 16), (n, 1, 1, 16), (1, n, 1, 16)):
        q = x.expand(shape)
        with pytest.raises(ValueError, match="2\\^31"):
            ttt._attn_desc(q, q, q, torch.zeros(1), None, None, 1.0, q)
        with pytest.raises(ValueError, match="2\\^31"):
            ttt._rotary_desc(q, q, q, q, 0)
        with pytest.raises(ValueError, match="2\\^31"):
            ttt.linear_attn_workspace_bytes(q, q)


def test_positions_are_whole_and_fit():
    q, f = torch.zeros(1, 1, 3, 16), torch.ones(8, dtype=torch.float64)
    check, ttt._check_same_dev = ttt._check_same_dev, lambda *a: None
    try:
        assert ttt._rope(q, 7, f).pos_offset == 7 and ttt._rope(q, -(1 << 40), f).pos_offset == -(1 << 40)
        for bad in (1 << 63, -(1 << 63) - 1):
            with pytest.raises(ValueError, match="position"):
                ttt._rope(q, bad, f)
        with pytest.raises(ValueError, match="position"):
            ttt._rope(q, 1.5, f)
    finally:
        ttt._check_same_dev = check
