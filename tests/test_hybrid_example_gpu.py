"""The example of a hybrid model's layers from prompts to log probabilities, on a GPU."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompts", [(200, 63, 130), (64, 1, 129)])
def test_prompts_trees_and_tokens(prompts):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import oracle
    import tree_speculative_verify_tv_gb300 as tv
    from examples import hybrid_serving
    tv.build()
    oracle.build()
    # run() holds every result to its bar: 2e-3 of a row's largest value, the library's parity
    # bar, and half a bf16 step for the rotated rows
    assert hybrid_serving.run(prompts=prompts) <= 2.0 ** -8 + 2.0 ** -16
