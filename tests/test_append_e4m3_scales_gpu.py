"""qk_norm_rope_paged on pages in 8 bits whose scale a caller chose: 0 over codes
that are not, and numbers that are no powers of two, on the GPU against the oracle (tolerances: test_append_e4m3_gpu.Append.check)."""
import numpy as np
import pytest

import oracle.paged_e4m3 as ref
import transformer_head_scaled_03_gb300 as mha
from transformer_head_scaled_03_gb300 import build as mha_build
from transformer_head_scaled_03_gb300.inputs import round_to_bf16
from tests.gpu_util import to_np
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


def twice(x):
    """x rounded to fp32 and then to e4m3, where once is meant."""
    return ref.encode(x.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("lens,new", FORMS)
@pytest.mark.parametrize("ps,d", [(16, 64), (256, 128)])
def test_quotients_by_any_scale_are_rounded_once(lens, new, ps, d):
    """Scales that are no powers of two, and values whose quotients are ties of
    e4m3 numbers or so near one that fp32 cannot tell."""
    ties = [(k, m * k) for k in (3, 5, 7) for m in range(17, 32, 2) if m * k < 256]
    near = [(np.nextafter(np.float32(1.875), np.float32(s)), v) for s in (1, 2) for v in (255, 240, 225)]
    near += [(np.nextafter(np.float32(7), np.float32(s)), 7 * m) for s in (6, 8) for m in range(17, 32, 2)]
    x = Append(951, lens, new, 4, 2, ps, d, 64, mha.ROPE_HALF)
    differ = 0
    for scale in sorted({np.float32(s) for s, _ in ties + near}):
        values = np.array([v for s, v in ties + near if np.float32(s) == scale], np.float32)
        with np.errstate(all="ignore"):
            differ += np.sum(twice(values * (np.float32(1) / scale)) != ref.encode(values / np.float64(scale)))
        x.vs[:] = scale
        x.v[...] = values[np.arange(x.v.size).reshape(x.v.shape) % len(values)]
        x.v[..., 1::2] *= -1
        state = x.state()
        x.run(state)
        assert mha.mha_check() == mha.MHA_OK
        x.check(state)
    assert differ >= 3


@pytest.mark.parametrize("lens,new", FORMS)
@pytest.mark.parametrize("ps,d", [(16, 64), (256, 128)])
def test_older_rows_are_rounded_once(lens, new, ps, d):
    """A page's scale that is no power of two grows to one that is."""
    x = Append(952, lens, new, 4, 2, ps, d, 64, mha.ROPE_HALF)
    x.v[...] = round_to_bf16(x.v * np.float32(512))
    codes = np.arange(127)                  # of numbers of either sign
    for c, m in ((9, 29), (9, 31), (11, 23), (11, 31), (13, 19), (13, 23), (15, 19), (15, 27)):
        old = np.float32(m / c)             # c * old is nearly, but not quite, m
        exact = ref.VALUES[:127] * np.float64(old) / 8
        assert np.sum(twice(exact) != ref.encode(exact)) >= 12
        x.vs[:] = x.ks[:] = old
        x.vc[:] = codes[np.arange(x.vc.size).reshape(x.vc.shape) % 127]
        x.vc[..., 1::3] |= 128
        state = x.state()
        x.run(state)
        assert mha.mha_check() == mha.MHA_OK
        grown = [x.table[b, (n - k) // ps] for b, (n, k) in enumerate(zip(lens, new)) if (n - k) % ps]
        assert np.all(to_np(state[3])[grown] >= 4)
        x.check(state)
