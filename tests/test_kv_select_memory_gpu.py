"""What kv_pages_select's results hold in device memory."""
import numpy as np
import pytest
import torch

import oracle.paged_e4m3 as ref
import transformer_head_scaled_03_gb300 as mha
from transformer_head_scaled_03_gb300 import build as mha_build
from tests.test_kv_select_gpu import run_select, select_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    mha_build.build()
    mha.lib()


@pytest.mark.parametrize("cols", [700, 300000])
def test_selections_do_not_hold_the_scores(cols):
    """The workspace, a score for every column of the table, goes back when the
    call's stream is past it, but for a small one's."""
    x = select_case(970, [500, 300], [3, 2], 4, 2, 16, 64, cols=cols)
    want, rows = ref.select(x[0], *x[1:], 5)
    scores = mha.lib().kv_pages_select_workspace_bytes(5, 2, cols)
    sel, got = run_select(x, 5)
    assert mha.mha_check() == mha.MHA_OK
    assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(got.cpu().numpy(), rows)
    held = sel.untyped_storage().nbytes()
    assert held == got.untyped_storage().nbytes()
    assert held <= 4 * (sel.numel() + got.numel()) + 16 + min(scores, 8 << 20)
    if scores > 8 << 20:
        assert held < scores
    for stream in (None, torch.cuda.Stream()):
        again = run_select(x, 5, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(again[0], sel) and torch.equal(again[1], got)
