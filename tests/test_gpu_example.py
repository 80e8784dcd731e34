"""The example that runs the product and the attention operators together."""
import os
import runpy

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_prompt_and_drafts(capsys):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from all_gather_gemm_agmm_gb300 import _build

    _build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "prompt_and_drafts.py")
    runpy.run_path(path, run_name="__main__")
    assert "trees" in capsys.readouterr().out
