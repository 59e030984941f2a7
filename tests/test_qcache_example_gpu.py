"""The example of the 4-bit KV cache in the speculation loop, on a GPU."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompts", [(200, 63, 1), (64, 0, 129)])
def test_the_loop_over_a_quantised_cache(prompts):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import oracle
    import tree_speculative_verify_tv_gb300 as tv
    from examples import qcache_step
    tv.build()
    oracle.build()
    # the oracle's values are the kernel's inputs exactly; what differs is fp32 sums and
    # exponentials and the weights' two or three bf16 parts: far below the bar of 2e-3
    assert qcache_step.run(prompts=prompts) <= 2e-3
