"""Bad offsets and lengths given to kv_pages_select, on the GPU: all of them are
reported, whether or not a token resolves to them."""
import numpy as np
import pytest

import transformer_head_scaled_03_gb300 as mha
from transformer_head_scaled_03_gb300 import build as mha_build
from tests.test_kv_select_gpu import run_select, select_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    mha_build.build()
    mha.lib()


def status(x, n=3, **kw):
    y = list(x)
    for k, v in kw.items():
        y[dict(lens=3, offs=4)[k]] = np.asarray(v, np.int32)
    run_select(y, n)
    return mha.mha_check()


@pytest.mark.parametrize("offs", [[0, 5, 3, 8], [0, 8, 8, 7], [2, 0, 4, 8], [-1, 3, 4, 8], [0, 9, 9, 8],
                                  [0, 2, 3, 2 ** 31 - 1], [0, 2, -2 ** 31, 8]])
def test_offsets_that_descend_or_leave_the_tokens(offs):
    x = select_case(960, [100, 90, 300], [3, 2, 3], 2, 1, 16, 64)
    assert status(x) == mha.MHA_OK
    assert status(x, offs=offs) == mha.MHA_ERR_DEVICE
    assert status(x) == mha.MHA_OK


@pytest.mark.parametrize("B,at", [(3, 2), (70, 0), (70, 33), (300, 299)])
def test_one_bad_sequence_of_many(B, at):
    lens, new = [40] * B, [1] * B
    x = select_case(961, lens, new, 2, 1, 16, 64)
    assert status(x) == mha.MHA_OK
    for n in (0, -7, 49):
        bad = np.array(lens)
        bad[at] = n
        assert status(x, lens=bad) == mha.MHA_ERR_DEVICE
    # of a sequence without new tokens the length is not looked at
    idle = np.concatenate((np.arange(at + 1), np.arange(at, B)))
    bad = np.array(lens)
    bad[at] = -7
    assert status(x, offs=idle, lens=bad) == mha.MHA_OK
    offs = np.arange(B + 1)
    offs[at + 1] = B + 1
    assert status(x, offs=offs) == mha.MHA_ERR_DEVICE
