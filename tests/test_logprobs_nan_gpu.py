"""tv_logprobs: a NaN counts as the largest logit wherever it stands, the first of a row too."""
import numpy as np
import pytest

import oracle
import workloads
from test_logprobs_gpu import call, check, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()


@pytest.mark.parametrize("V", [1, 2, 20, 32, 33, 1003, 40000])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("R", [6, 400])
def test_nan_at_the_first_token(V, f32, R):
    """R = 6: long rows are cut over clusters; 400: a CTA has a whole row."""
    rng = np.random.default_rng(1)
    x = values(rng, (6, V), f32)
    x[0, 0] = np.nan
    x[1] = np.nan
    x[2, [0, V // 2, V - 1]] = np.nan
    x[3, 0], x[3, V - 1] = np.nan, np.inf
    x[4, V - 1] = np.nan
    x[5] = -np.inf
    x[5, 0] = np.nan
    x = np.concatenate([x] * (-(-R // 6)))[:R]
    tokens = rng.integers(0, V, R)
    top = min(V, 32)
    got = call(x, f32, None, tokens, 1.0, top)
    check(x, f32, None, tokens, 1.0, top, got)
    if not f32:
        assert np.array_equal(got[2][:, 0], oracle.argmax_rows(workloads.f32_to_bf16_bits(x)))


def test_nan_of_any_sign_and_payload():
    """All bit patterns that are NaNs are alike: the lower index first."""
    bits = np.zeros((2, 50), np.uint32)
    bits[0, [0, 3, 9, 30]] = 0xFFFFFFFF, 0x7FC00000, 0x7FFFFFFF, 0xFF800001
    bits[1, [7, 8]] = 0x7FFFFFFE, 0xFFC00000
    x = bits.view(np.float32)
    top = call(x, True, None, None, 1.0, 5)[2]
    assert top.tolist() == [[0, 3, 9, 30, 1], [7, 8, 0, 1, 2]]
