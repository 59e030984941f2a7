"""One slow decay over many rows: what a row's decay is rounded to does not add up."""
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


@pytest.mark.parametrize("workspace", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_a_slow_decay_over_65536_rows(d, workspace):
    """States that begin at order 1, to which rows add 1/8 at most in all.  Normwise: 1024 chunks
    round the state once each (2^-24, independent of each other), and twice the norm of their sum
    is allowed; sums of what is added are off by at most 28 roundings (2^-24) of 1/8 of a state.
    A row's decay cut to a multiple of 2^-32 log2 units would be off by 0.93 to 0.95 of that,
    always the same way: 65536 rows of it are 1e-5 of the state, 2.4 times the bound."""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    n, gates = 65536, (-9.002e-07, -1.7081e-06, -2.4792e-06)
    fixed = np.abs(np.array(gates, np.float32).astype(np.float64)) / np.log(2) * 2.0 ** 32
    assert ((fixed % 1 > 0.92) & (fixed % 1 < 0.96)).all()
    H = len(gates)
    gen = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = (torch.randn(n, H, d, generator=gen, device="cuda") for _ in range(3))
    scale = 0.125 / n ** 0.5  # (|k| |v| n is 1/8 of an element of the state, and less in the mean)
    q, k, v = q.bfloat16(), (k * scale).bfloat16(), (v * n ** -0.5).bfloat16()
    g = torch.tensor(gates, device="cuda")
    H0 = torch.randn(1, H, d, d, generator=gen, device="cuda")
    H_new, out = torch.empty_like(H0), torch.empty(n, H, d, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    size = (tv.tv_prefill_workspace_bytes(1, n, n, H, d, d, tv.TV_DECAY_SCALAR, tv.TV_BF16)
            if workspace else 0)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    tv.tv_prefill(1, n, n, H, d, d, tv.TV_DECAY_SCALAR, tv.TV_BF16, offsets, H0, q, H * d, k, H * d, v,
                  H * d, g, 0, tv.TV_F32, out, H_new, ws, size, status)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    age = torch.arange(n - 1, -1, -1, device="cuda", dtype=torch.float64)
    w = torch.exp(age[:, None] * g.double()[None])
    want = (torch.exp(n * g.double())[:, None, None] * H0[0].double() +
            torch.einsum("thc,thd->hcd", k.double() * w[..., None], v.double()))
    bound = 2 * 2.0 ** -24 * np.sqrt(n / 64) + 28 * 2.0 ** -24 / 8
    for h in range(H):
        err = float((H_new[0, h].double() - want[h]).norm() / want[h].norm())
        assert err <= bound, (gates[h], err, bound)
