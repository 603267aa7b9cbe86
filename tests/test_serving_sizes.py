"""Sizes the serving binding takes on the host (CPU only)."""
import pytest

pytest.importorskip("torch")

import block_text_diffusion_b200 as dg  # noqa: E402


def test_workspace_sizes_past_32_bits_are_refused():
    from block_text_diffusion_b200 import build
    build.build()
    assert dg.paged_attention_workspace(5, 4, 128) > 0
    for args in (((1 << 32) + 5, 4, 128), (5, (1 << 32) + 4, 128), (5, 4, (1 << 32) + 128), (-(1 << 32) + 5, 4, 128),
                 (-1, 4, 128)):
        with pytest.raises(dg.DGError):
            dg.paged_attention_workspace(*args)
