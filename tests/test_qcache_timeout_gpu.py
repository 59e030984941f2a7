"""The timeout path of the attention over the 4-bit cache: with the test hook every CTA's first
unit is left unprepared, what waits for it gives up, and the call ends with TV_ERR_TIMEOUT after
its copies and products in flight; the next ordinary call on the same stream is exact."""
import time

import numpy as np
import pytest

from tests.test_qcache_gpu import attend, check_rows, cu, make, status, strided

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,nodes,H", [(64, 1, 4), (128, 1, 4), (64, 40, 4), (128, 40, 4)])
@pytest.mark.parametrize("half", [False, True])
def test_timeout_then_an_ordinary_call(d, nodes, H, half):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()
    # more tiles per CTA than the ring and the operand buffers hold, and more units than the
    # ring of segments: every role is stopped in the middle
    B, Hkv = 40, 2
    ctx = [64 * (3 + b % 7) for b in range(B)]
    ctx[0] = 5000
    b, c = make(d + nodes, [nodes] * B, Hkv, d, ctx)
    rng = np.random.default_rng(1)
    rows = strided(rng, b.T, [H * d, Hkv * d, Hkv * d], 0)
    s, good, args = attend(c, b, ctx, H, half=half, rows=rows)
    assert s == 0
    ((q, _), (kt, _), (vt, _)), stride = rows
    kind = tv.TV_BF16 if half else tv.TV_F32
    out = torch.zeros((b.T, H, d), device="cuda", dtype=torch.bfloat16 if half else torch.float32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    size = tv.tv_qcache_attention_workspace_bytes(B, b.T, b.max_nodes, H, Hkv, d, c.mp)
    ws = torch.zeros(max(size, 16), dtype=torch.uint8, device="cuda")
    offs, par, lens = cu(b.node_offsets), cu(b.parent), cu(np.asarray(ctx, np.int32))

    def call(kind):
        tv.tv_qcache_attention(B, b.T, b.max_nodes, H, Hkv, d, c.pages, c.mp, offs, par, lens,
                               c.dev_table, 0, 0, q, stride, c.dev, kt, vt, stride, d ** -0.5, kind, out,
                               ws, size, st)

    torch.cuda.synchronize()
    t = time.monotonic()
    call(kind | tv.TV_QCACHE_TEST_EXPIRE_WAIT)
    assert status(st) == tv.TV_ERR_TIMEOUT
    assert time.monotonic() - t < 2
    for _ in range(2):
        st.zero_()
        out.fill_(float("nan"))
        call(kind)
        assert status(st) == 0
        assert np.array_equal(out.float().cpu().numpy(), good)
    check_rows(good, *args)
