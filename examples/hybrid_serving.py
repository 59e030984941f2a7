"""A hybrid model's two kinds of layers from the prompt to the answer's log probabilities.

    prompts: recurrence layer  tv_prefill -> the state that the trees are verified from
             attention layer   tv_qk_norm_rope -> tv_qcache_write
    a step:  recurrence layer  tv_verify of the draft trees
             attention layer   tv_qk_norm_rope at the nodes' positions -> tv_qcache_attention
             logits            tv_accept_greedy_logits, tv_logprobs of what it emits
             commit            tv_commit, tv_qcache_commit
    a token: tv_decode, and the attention layer's tree of one node

run() checks every result against the fp64 oracle and returns the worst relative error.
    python examples/hybrid_serving.py
"""
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import oracle  # noqa: E402
import workloads  # noqa: E402

HR, DK, DV = 3, 128, 64                # the recurrence layer's heads and widths
H, HKV, D, MAX_PAGES = 8, 2, 128, 6    # the attention layer's, and pages per request
SCALE, EPS, VOCAB, TOP = D ** -0.5, 1e-6, 1003, 4
FREQ = 10000.0 ** (-np.arange(0, D, 2) / D)


def run(prompts=(200, 63, 130), steps=2, seed=21) -> float:
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    rng = np.random.default_rng(seed)
    B = len(prompts)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    worst = [0.0]

    def near(got, want, bar=2e-3):
        """Row by row: the largest difference against the row's largest value."""
        got = got.float().cpu().numpy().astype(np.float64).reshape(want.shape)
        if not want.size:
            return
        err = np.abs(got - want).max(-1) / np.maximum(np.abs(want).max(-1), 1e-30)
        assert err.max() <= bar, "relative error %.3e" % err.max()
        worst[0] = max(worst[0], float(err.max()))

    def projected(n, **heads):
        """Rows of one fused projection: device views, their row stride, and their values."""
        widths = [h * d for h, d in heads.values()]
        x = (rng.normal(size=(n, sum(widths))) * 0.3).astype(np.float32)
        bits = workloads.f32_to_bf16_bits(x)
        parts = dev(bits).view(torch.bfloat16).split(widths, 1)
        cuts = np.split(workloads.bf16_bits_to_f32(bits).astype(np.float64), np.cumsum(widths)[:-1], 1)
        return parts, sum(widths), [c.reshape(n, h, d) for c, (h, d) in zip(cuts, heads.values())]

    def gates(n):
        return (-np.logaddexp(0, rng.normal(-1, 0.5, (n, HR)))).astype(np.float32)

    # a rotation's norms: one weight per channel of a head
    wq, wk = (workloads.bf16_bits_to_f32(workloads.f32_to_bf16_bits(
        (1 + 0.1 * rng.normal(size=D)).astype(np.float32))) for _ in range(2))
    dwq, dwk = (dev(w).to(torch.bfloat16) for w in (wq, wk))
    freq = dev(FREQ)

    def rotated(offsets, start, depth, q, k, stride, hq, hk):
        """tv_qk_norm_rope into packed rows; the values that it should give."""
        n = int(offsets[-1])
        qo, ko = new(n, H * D, dtype=torch.bfloat16), new(n, HKV * D, dtype=torch.bfloat16)
        first = start.cpu().numpy().astype(np.int64)
        tv.tv_qk_norm_rope(B, n, H, HKV, D, D, tv.TV_ROPE_HALVES, tv.TV_BF16, dev(offsets), start,
                           None if depth is None else dev(depth), q, stride, k, stride, dwq, dwk,
                           EPS, freq, qo, H * D, ko, HKV * D, status)
        b = np.repeat(np.arange(B), np.diff(offsets))
        pos = first[b] + (np.arange(n) - offsets[b] if depth is None else depth - 1)
        for x, hx, w in ((qo, hq, wq), (ko, hk, wk)):
            # bf16: half a step, 2^-8 of a value, whose row's largest is no smaller
            near(x, oracle.qk_norm_rope(hx, pos, w, EPS, FREQ, False), 2.0 ** -8 + 2.0 ** -16)
        return qo, ko, [x.float().cpu().numpy().astype(np.float64).reshape(n, -1, D) for x in (qo, ko)]

    # ---- the prompts
    at = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
    R, most = int(at[-1]), max(prompts)
    (q, k, v), stride, host = projected(R, q=(HR, DK), k=(HR, DK), v=(HR, DV))
    g = gates(R)
    out, state = new(R, HR, DV), new(B, HR, DK, DV)
    nb = tv.tv_prefill_workspace_bytes(B, R, most, HR, DK, DV, tv.TV_DECAY_SCALAR, tv.TV_BF16)
    ws = new(max(nb, 16), dtype=torch.uint8)
    tv.tv_prefill(B, R, most, HR, DK, DV, tv.TV_DECAY_SCALAR, tv.TV_BF16, dev(at), None, q, stride,
                  k, stride, v, stride, dev(g), HR, tv.TV_F32, out, state, ws, nb, status)
    want, S = oracle.prefill(at, *host, g)
    near(out, want)
    near(state.flatten(2), S.reshape(B, HR, -1))

    table, pages = workloads.qcache_pages(rng, B, MAX_PAGES)
    cache = torch.zeros(tv.tv_qcache_bytes(pages, HKV, D), dtype=torch.uint8, device="cuda")
    dtable, ctx, zero = dev(table), dev(np.array(prompts, np.int32)), dev(np.zeros(B, np.int32))
    (q, k, v), stride, (hq, hk, hv) = projected(R, q=(H, D), k=(HKV, D), v=(HKV, D))
    _, ko, (_, kv) = rotated(at, zero, None, q, k, stride, hq, hk)
    vo = v.contiguous()  # (one stride serves the cache's keys and values)
    tv.tv_qcache_write(B, R, HKV, D, pages, MAX_PAGES, dev(at), zero, dtable, ko, vo, HKV * D, cache,
                       status)
    quantised = lambda x: oracle.qcache_values(*oracle.qcache_quantise(x)) if len(x) else x  # noqa: E731
    held = [[quantised(x[at[b]:at[b + 1]]) for b in range(B)] for x in (kv, hv)]

    def attention(offsets, parent, depth, max_nodes):
        n = int(offsets[-1])
        (q, k, v), stride, (hq, hk, hv) = projected(n, q=(H, D), k=(HKV, D), v=(HKV, D))
        qo, ko, (qv, kv) = rotated(offsets, ctx, depth, q, k, stride, hq, hk)
        vo, o = v.contiguous(), new(n, H, D)
        nb = tv.tv_qcache_attention_workspace_bytes(B, n, max_nodes, H, HKV, D, MAX_PAGES)
        ws = new(max(nb, 16), dtype=torch.uint8)
        tv.tv_qcache_attention(B, n, max_nodes, H, HKV, D, pages, MAX_PAGES, dev(offsets),
                               dev(parent), ctx, dtable, 0, 0, qo, H * D, cache, ko, vo, HKV * D,
                               SCALE, tv.TV_F32, o, ws, nb, status)
        full = [np.zeros((B, HKV, MAX_PAGES * 64, D)) for _ in range(2)]
        for x, h in zip(full, held):
            for b in range(B):
                x[b, :, :len(h[b])] = h[b].transpose(1, 0, 2)
        near(o, oracle.qcache_attention(offsets, parent, qv, *full, ctx.cpu().numpy(), kv, hv, SCALE,
                                        0, 0))
        return ko, vo, kv, hv

    # ---- steps over draft trees
    for _ in range(steps):
        b = workloads.random_batch(rng, [9, 4, 16][:B], HR, DK, DV, depth_cap=5, max_depth=8,
                                   vocab=VOCAB)
        b.H0 = state.cpu().numpy()
        d = tv.DeviceBatch(b)
        d.H0.copy_(state)
        d.status.zero_()
        d.verify()
        for u, ref in oracle.verify(b).items():
            r, h = divmod(u, HR)
            near(d.out[b.node_offsets[r]:b.node_offsets[r + 1], h], ref)
        ko, vo, kv, hv = attention(b.node_offsets, b.parent, b.depth, b.max_nodes)

        # logits of the context rows, then of the nodes'; the walk, and what it emits
        rl, nl = workloads.target_logits(b, VOCAB, seed=int(rng.integers(1 << 30)))
        logits = dev(np.concatenate([rl, nl])).view(torch.bfloat16)
        nodes = logits[B:].clone()  # (row B of an odd vocabulary is not 16-byte aligned)
        ra, ta = new(B, dtype=torch.int32), new(b.T, dtype=torch.int32)
        tv.tv_accept_greedy_logits(B, b.T, b.max_nodes, b.max_depth, VOCAB, d.node_offsets, d.parent,
                                   d.draft, logits[:B], nodes, ra, ta, d.accept_len, d.path, d.bonus,
                                   status)
        # emitted tokens of a request: the accepted nodes' drafts, then the bonus token; each
        # stands under the row before it, the context's or the node's before
        path, first = d.path.long(), d.node_offsets[:-1, None].long()
        node = torch.where(path >= 0, first + path, -1)
        after = torch.cat([torch.arange(B, device="cuda")[:, None],
                           torch.where(node >= 0, B + node, -1)], 1)
        L = d.accept_len[:, None].long()
        slot = torch.arange(after.shape[1], device="cuda")[None]
        drafts = torch.where(node >= 0, d.draft[node.clamp(min=0)].long(), -1)
        emitted = torch.cat([drafts, torch.full_like(L, -1)], 1)
        emitted = torch.where(slot == L, d.bonus[:, None].long(), emitted)
        rows = torch.where(slot <= L, after, -1).int().flatten().contiguous()
        tokens = emitted.int().flatten().contiguous()
        n = rows.numel()
        lp, ent, tt, tl = new(n), new(n), new(n, TOP, dtype=torch.int32), new(n, TOP)
        tv.tv_logprobs(n, B + b.T, VOCAB, tv.TV_BF16, logits, VOCAB, rows, tokens, 1.0, TOP, lp, ent,
                       tt, tl, status)
        ln, hp, _ = oracle.accept_batch(b)
        assert np.array_equal(d.accept_len.cpu().numpy(), ln)
        want = oracle.logprobs(workloads.bf16_bits_to_f32(np.concatenate([rl, nl])),
                               rows.cpu().numpy(), tokens.cpu().numpy(), 1.0, TOP)
        assert np.array_equal(tt.cpu().numpy(), want[2])
        # an emitted token is the greedy choice of its row
        live = rows.cpu().numpy() >= 0
        assert np.array_equal(want[2][live, 0], tokens.cpu().numpy()[live])
        for x, y in ((lp, want[0]), (ent, want[1]), (tl, want[3])):
            assert np.abs(x.cpu().numpy() - y).max() <= 1e-5

        # the accepted paths
        d.commit(in_place=True)
        for u, ref in oracle.commit(b, ln, hp).items():
            near(d.H0[u // HR, u % HR].flatten(), ref.flatten())
        state = d.H0
        tv.tv_qcache_commit(B, b.T, b.max_nodes, b.max_depth, HKV, D, pages, MAX_PAGES,
                            d.node_offsets, d.path, d.accept_len, ctx, dtable, ko, vo, HKV * D,
                            cache, ctx, status)
        for r in range(B):
            picked = b.node_offsets[r] + hp[r, :ln[r]]
            for h, x in zip(held, (kv, hv)):
                h[r] = np.concatenate([h[r], quantised(x[picked])])
        assert int(d.status[0]) == 0, tv.status_string(int(d.status[0]))

    # ---- one token of every request, without drafts
    (q, k, v), stride, host = projected(B, q=(HR, DK), k=(HR, DK), v=(HR, DV))
    g, out = gates(B), new(B, HR, DV)
    H0 = state.cpu().numpy()
    tv.tv_decode(B, HR, DK, DV, tv.TV_DECAY_SCALAR, tv.TV_BF16, None, state, q, stride, k, stride, v,
                 stride, dev(g), HR, tv.TV_F32, out, state)
    want, S = oracle.prefill(np.arange(B + 1), *host, g, H0)
    near(out, want)
    near(state.flatten(2), S.reshape(B, HR, -1))
    attention(np.arange(B + 1, dtype=np.int32), np.full(B, -1, np.int32), np.ones(B, np.int32), 1)

    assert int(status[0]) == 0, tv.status_string(int(status[0]))
    return worst[0]


if __name__ == "__main__":
    import tree_speculative_verify_tv_gb300
    tree_speculative_verify_tv_gb300.build()
    oracle.build()
    print("worst relative error %.2e" % run())
