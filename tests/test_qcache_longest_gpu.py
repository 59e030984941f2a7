"""A unit that one CTA works on for seconds is not taken for one that hangs."""
import pytest

pytestmark = pytest.mark.gpu


def test_three_quarters_of_a_billion_positions():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()
    # 152 units of 64 rows over 3 * 2^28 positions (one page, over and over): seconds, of which the warps
    # that prepare a CTA's second unit wait all
    d, H, nodes, ctx = 64, 128, 76, 3 << 28
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = torch.randint(0, 128, (tv.tv_qcache_bytes(1, 1, d),), dtype=torch.uint8, device="cuda")
    table = torch.zeros(ctx // 64, dtype=torch.int32, device="cuda")
    q = torch.randn(nodes, H, d, device="cuda").bfloat16()
    kv = torch.randn(nodes, d, device="cuda").bfloat16()
    out = torch.empty(nodes, H, d, dtype=torch.bfloat16, device="cuda")
    size = tv.tv_qcache_attention_workspace_bytes(1, nodes, nodes, H, 1, d, ctx // 64)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    st = i32([0])
    tv.tv_qcache_attention(1, nodes, nodes, H, 1, d, 1, ctx // 64, i32([0, nodes]),
                           i32(list(range(-1, nodes - 1))), i32([ctx]), table, 0, 0, q, H * d, cache,
                           kv, kv, d, 0.1, tv.TV_BF16, out, ws, size, st)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    assert bool(torch.isfinite(out).all())
