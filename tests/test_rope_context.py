"""The frequencies' scalings that go by the trained context are not guessed without one."""
import pytest
import torch


def test_context_is_asked_for(epq_lib):
    e = epq_lib
    for kind in (e.EPQ_ROPE_PARTS, e.EPQ_ROPE_BANDS):
        with pytest.raises(ValueError):
            e.epq_rope_frequencies(128, 500000.0, kind, 8.0)
        with pytest.raises(ValueError):
            e.RopeTable(128, 16, 500000.0, device="cpu", kind=kind, factor=8.0)
        e.epq_rope_frequencies(128, 500000.0, kind, 8.0, 1.0)
    plain, _ = e.epq_rope_frequencies(128, 500000.0)
    linear, _ = e.epq_rope_frequencies(128, 500000.0, e.EPQ_ROPE_LINEAR, 8.0)
    assert torch.equal(plain, linear * 8.0)
