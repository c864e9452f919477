"""The long-context example runs in every format and keeps to its budget (GPU)."""
import os
import sys

import pytest
import torch

import mixture_experts_gb300 as moe

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4", "f32"])
def test_long_context(fmt, capsys):
    moe.build()
    import long_context
    chats = long_context.main(["--format", fmt, "--batch", "9", "--prompt", "301", "--budget", "40",
                               "--steps", "75"])
    assert (chats.lens <= 40 + 16).all() and (chats.lens >= 40).all()
    assert fmt in capsys.readouterr().out
    assert torch.isfinite(chats.mass).all()
