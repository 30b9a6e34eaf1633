"""qk_norm_rope_paged on pages in 8 bits whose scale a caller chose: 0 over codes
that are not, on the GPU against the oracle (tolerances: test_append_e4m3_gpu.Append.check)."""
import numpy as np
import pytest

import transformer_head_scaled_03_gb300 as mha
from transformer_head_scaled_03_gb300 import build as mha_build
from tests.test_append_e4m3_gpu import Append

pytestmark = pytest.mark.gpu

# a warp to a page's rows; a block
FORMS = [([37, 100, 18], [1, 1, 2]), ([45, 300, 18], [20, 130, 1])]


@pytest.fixture(scope="module", autouse=True)
def built():
    mha_build.build()
    mha.lib()


@pytest.mark.parametrize("lens,new", FORMS)
@pytest.mark.parametrize("ps,d", [(16, 64), (64, 128), (256, 64)])
def test_rows_under_a_scale_of_zero_stay_zeros(lens, new, ps, d):
    """Codes of any kind under a scale of 0 are rows of zeros; new rows give the
    page a scale, and the older ones are zeros under it too."""
    x = Append(950, lens, new, 4, 2, ps, d, 64, mha.ROPE_HALF)
    older = [x.table[b, (n - m) // ps] for b, (n, m) in enumerate(zip(lens, new)) if (n - m) % ps]
    assert older and all(np.any(x.kc[p] & 127) for p in older)
    x.ks[older], x.vs[older] = 0, 0
    state = x.state()
    x.run(state)
    assert mha.mha_check() == mha.MHA_OK
    x.check(state)
