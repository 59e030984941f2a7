"""An attention layer of the speculation loop over a paged 4-bit KV cache.

    prompt -> tv_qcache_write
    each step:  tv_qcache_attention over the draft trees (their nodes' own bf16 rows beside
                the cache), tv_accept_greedy, tv_qcache_commit of the accepted nodes' rows
    at the end: tv_qcache_read of the last positions, and one decoding step of a layer with
                a sliding window and sinks (a tree of one node per request)

run() checks every result against the fp64 oracle and returns the worst relative error.
    python examples/qcache_step.py
"""
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import oracle  # noqa: E402
import workloads  # noqa: E402

HKV, H, D, MAX_PAGES = 2, 8, 128, 6
SCALE = D ** -0.5


def run(prompts=(200, 63, 1), steps=2, seed=11) -> float:
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    rng = np.random.default_rng(seed)
    B = len(prompts)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rows(n, heads):  # n rows of bf16 on the device, and their values
        bits = workloads.f32_to_bf16_bits(rng.normal(size=(n, heads * D)).astype(np.float32))
        return (dev(bits).view(torch.bfloat16),
                workloads.bf16_bits_to_f32(bits).reshape(n, heads, D).astype(np.float64))

    # the cache: pages of 64 positions, a table of them per request, lengths on the device
    table, pages = workloads.qcache_pages(rng, B, MAX_PAGES)
    cache = torch.zeros(tv.tv_qcache_bytes(pages, HKV, D), dtype=torch.uint8, device="cuda")
    dtable, ctx = dev(table), dev(np.array(prompts, np.int32))
    held = [[], []]  # what the cache should hold: K, V rows per request, as values

    def quantised(x):  # the values that rows x [n][HKV][D] read back as
        return oracle.qcache_values(*oracle.qcache_quantise(x)) if len(x) else x

    def check_cached():
        """The cache's positions read back, against the rows that went in."""
        lens = [len(k) for k in held[0]]
        offs = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
        k, v = (torch.empty((sum(lens), HKV * D), dtype=torch.bfloat16, device="cuda")
                for _ in range(2))
        tv.tv_qcache_read(B, sum(lens), HKV, D, pages, MAX_PAGES, offs,
                          dev(np.zeros(B, np.int32)), ctx, dtable, cache, k, v, HKV * D, status)
        for x, want in zip((k, v), held):
            got = x.float().cpu().numpy().reshape(-1, HKV, D)
            assert np.array_equal(got, np.concatenate(want)), "cache contents"
        assert ctx.cpu().tolist() == lens, "lengths"

    def attention(offsets, parent, max_nodes, window, sinks, out_dtype):
        """One layer's attention of a batch of trees: its error, and the trees' K, V rows."""
        T = int(offsets[-1])
        (q, qv), (k, kv), (v, vv) = rows(T, H), rows(T, HKV), rows(T, HKV)
        out = torch.empty((T, H, D), device="cuda",
                          dtype=torch.float32 if out_dtype == tv.TV_F32 else torch.bfloat16)
        nb = tv.tv_qcache_attention_workspace_bytes(B, T, max_nodes, H, HKV, D, MAX_PAGES)
        ws = torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda")
        tv.tv_qcache_attention(B, T, max_nodes, H, HKV, D, pages, MAX_PAGES, dev(offsets),
                               dev(parent), ctx, dtable, window, sinks, q, H * D, cache, k, v,
                               HKV * D, SCALE, out_dtype, out, ws, nb, status)
        full = [np.zeros((B, HKV, MAX_PAGES * 64, D)) for _ in range(2)]
        for x, h in zip(full, held):
            for b in range(B):
                x[b, :, :len(h[b])] = h[b].transpose(1, 0, 2)
        ref = oracle.qcache_attention(offsets, parent, qv, *full, ctx.cpu().numpy(), kv, vv, SCALE,
                                      window, sinks)
        got = out.float().cpu().numpy().astype(np.float64)
        err = np.abs(got - ref).max(axis=-1) / np.abs(ref).max(axis=-1)
        return float(err.max()), (k, kv), (v, vv)

    # the prompts
    (k, kv), (v, vv) = rows(sum(prompts), HKV), rows(sum(prompts), HKV)
    at = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
    tv.tv_qcache_write(B, sum(prompts), HKV, D, pages, MAX_PAGES, dev(at),
                       dev(np.zeros(B, np.int32)), dtable, k, v, HKV * D, cache, status)
    for h, x in zip(held, (kv, vv)):
        h.extend(quantised(x[at[b]:at[b + 1]]) for b in range(B))
    check_cached()

    worst = 0.0
    for _ in range(steps):
        b = workloads.random_batch(rng, [9, 4, 16][:B], 1, 64, 64, depth_cap=5)
        err, (k, kv), (v, vv) = attention(b.node_offsets, b.parent, b.max_nodes, 0, 0, tv.TV_F32)
        worst = max(worst, err)
        # (the target's tokens come from the rest of the model; here from the batch)
        length, bonus = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
        path = torch.zeros((B, b.max_depth), dtype=torch.int32, device="cuda")
        offs = dev(b.node_offsets)
        tv.tv_accept_greedy(B, b.T, b.max_nodes, b.max_depth, offs, dev(b.parent), dev(b.draft),
                            dev(b.target), dev(b.root_argmax), length, path, bonus, status)
        tv.tv_qcache_commit(B, b.T, b.max_nodes, b.max_depth, HKV, D, pages, MAX_PAGES, offs, path,
                            length, ctx, dtable, k, v, HKV * D, cache, ctx, status)
        n, p, _ = oracle.accept_batch(b)
        for r in range(B):
            new = b.node_offsets[r] + p[r, :n[r]]
            for h, x in zip(held, (kv, vv)):
                h[r] = np.concatenate([h[r], quantised(x[new])])
        check_cached()

    # a token per request, in a layer that sees 100 positions and the first 4
    err, _, _ = attention(np.arange(B + 1, dtype=np.int32), np.full(B, -1, np.int32), 1, 100, 4,
                          tv.TV_F32)
    worst = max(worst, err)
    assert int(status[0]) == 0, tv.status_string(int(status[0]))
    assert worst <= 2e-3, "attention over the 4-bit cache: %.3e" % worst
    return worst


if __name__ == "__main__":
    import tree_speculative_verify_tv_gb300
    tree_speculative_verify_tv_gb300.build()
    oracle.build()
    print("worst relative error %.2e" % run())
