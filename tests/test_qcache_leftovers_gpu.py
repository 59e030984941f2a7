"""A call's time does not depend on what earlier launches left in shared memory: units whose rows
do not fill a block of columns, after a launch whose queries were huge and after one whose
queries were zero."""
import pytest

pytestmark = pytest.mark.gpu


def attention(B, nodes, grp, d, ctx, factor):
    """A call over B requests (chains) and 8 KV heads, with queries of the given size."""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    Hkv, mp, dev = 8, ctx // 64, "cuda"
    H, T, pages = Hkv * grp, B * nodes, B * mp
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(dev)  # noqa: E731
    cache = torch.randint(0, 128, (tv.tv_qcache_bytes(pages, Hkv, d),), dtype=torch.uint8, device=dev)
    q = (torch.randn(T, H, d, device=dev) * factor).bfloat16()
    kv = torch.randn(T, Hkv, d, device=dev).bfloat16()
    offs, parent = i32(range(0, T + 1, nodes)), i32(list(range(-1, nodes - 1)) * B)
    table, lens = i32(range(pages)), i32([ctx] * B)
    out = torch.empty(T, H, d, dtype=torch.bfloat16, device=dev)
    st = torch.zeros(4, dtype=torch.int32, device=dev)
    size = tv.tv_qcache_attention_workspace_bytes(B, T, nodes, H, Hkv, d, mp)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device=dev)

    def call():
        tv.tv_qcache_attention(B, T, nodes, H, Hkv, d, pages, mp, offs, parent, lens, table, 0, 0, q,
                               H * d, cache, kv, kv, Hkv * d, 0.01, tv.TV_BF16, out, ws, size, st)
    return call, st


@pytest.mark.parametrize("d,nodes,grp,full", [(128, 1, 1, (1, 32)), (64, 1, 9, (1, 32)), (128, 3, 11, (2, 32)),
                                              (64, 2, 30, (2, 32))])
def test_time_does_not_depend_on_rows_that_are_not_there(d, nodes, grp, full):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    call, st = attention(64, nodes, grp, d, 2048, 1.0)
    best = []
    for factor in (0.0, 1e30):  # units of the same number of rows, all of them live
        before, _ = attention(64, *full, d, 2048, factor)
        times = []
        for _ in range(20):
            before()
            torch.cuda.synchronize()
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            call()
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end))
        best.append(min(times))
    assert int(st[0]) == 0
    assert best[1] < 1.15 * best[0], "%.1f and %.1f us" % (best[1] * 1e3, best[0] * 1e3)
