"""Thousands of single tokens: the decay is applied as precisely as in a prompt."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()


GATES = (-1e-4, -3e-5, -1e-5, -1e-6)


def inputs(n, d, diag):
    """n rows of a head per gate (constant over the rows), and the state after them in 64 bits."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(5)
    H = len(GATES)
    q, k, v = (torch.randn(n, H, d, generator=gen, device="cuda").bfloat16() for _ in range(3))
    g = torch.tensor(GATES, device="cuda")
    age = torch.arange(n - 1, -1, -1, device="cuda", dtype=torch.float64)
    w = torch.exp(age[:, None] * g.double()[None])  # [n][H]
    want = torch.einsum("thc,thd->hcd", k.double() * w[..., None], v.double())
    gates = g[:, None].expand(H, d).contiguous() if diag else g
    return q, k, v, gates, want


def check(H_new, want, n, parts):
    """Normwise.  A step rounds the state once, by at most 2^-24 of it, one way or the other as the
    random products fall (`parts` such roundings a step, counting those of what is added): the sum
    of n independent ones is at most sqrt(n) of one in norm, and twice that is allowed.  A decay
    rounded to single precision is off in the same direction every step, by 0.2 to 0.36 of 2^-24 for
    these gates: over the rows' ages that adds up to 1.5e-4 (the first) to 3e-4, four to eight times
    the bound."""
    bound = 2 * parts * 2.0 ** -24 * np.sqrt(n)
    for i in range(len(GATES)):
        err = float((H_new[i].double() - want[i]).norm() / want[i].norm())
        assert err <= bound, (GATES[i], err, bound)


@pytest.mark.parametrize("diag", [False, True])
def test_a_slow_constant_decay_over_many_tokens(diag):
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    n, d, H = 40000, 64, len(GATES)
    q, k, v, g, want = inputs(n, d, diag)
    state = torch.zeros(1, H, d, d, device="cuda")
    out = torch.empty(1, H, d, device="cuda")
    decay = tv.TV_DECAY_DIAG if diag else tv.TV_DECAY_SCALAR
    for t in range(n):
        tv.tv_decode(1, H, d, d, decay, tv.TV_BF16, None, state, q[t], H * d, k[t], H * d, v[t], H * d,
                     g, 0, tv.TV_F32, out, state)
    torch.cuda.synchronize()
    check(state[0], want, n, 1.5)


def test_a_prompt_of_the_same_rows_agrees():
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    n, d, H = 40000, 64, len(GATES)
    q, k, v, g, want = inputs(n, d, False)
    state = torch.empty(1, H, d, d, device="cuda")
    out = torch.empty(n, H, d, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    tv.tv_prefill(1, n, n, H, d, d, tv.TV_DECAY_SCALAR, tv.TV_BF16, offsets, None, q, H * d, k, H * d,
                  v, H * d, g, 0, tv.TV_F32, out, state, None, 0, status)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    check(state[0], want, n, 1.5)
