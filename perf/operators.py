"""The operators of the 4-bit KV cache, as cases that can be timed and compared.

Each case is one call (or the pair of calls that belong together) of the cache's
operators: rows quantised into the pages and read back, an accepted path committed and
the cache read back, positions read back, tree attention over the cache.  `run` computes
them in elementary torch operations, or, where `own` is set, through the library.

The cache: pages of 64 positions; per (page, KV head) one record of
    K codes [d/32][64][16 B], K scales [64][d/32], V codes [2][d][16 B], V scales [d/32][64].
32 channels of a position share one scale byte b: s = (8 + b % 8) * 2^(b / 8 - 25), 255 = NaN.
Codes are 4 bits, value = s * (code - 8); K's 16 bytes hold 32 channels of one position,
V's hold 32 positions of one channel, in 32-bit words of 8 elements, element 2p in nibble p
and element 2p + 1 in nibble p + 4.
"""
import math

import numpy as np
import torch

own = False

PAGE, GROUP = 64, 32
NIBBLE = [0, 4, 1, 5, 2, 6, 3, 7]  # nibble of a word that holds its element e


def listed():
    return [
        # a batch of prompts prefilled into the cache, and read back whole
        dict(name="write_prompts", op="write", B=16, Hkv=8, d=128, lo=4096, hi=4096, start=0, fused=False, mix=1),
        # chunks of ragged length appended at odd positions, rows taken out of a fused projection
        dict(name="write_ragged_chunks", op="write", B=32, Hkv=4, d=64, lo=1, hi=97, start=500, fused=True, mix=2),
        # the accepted paths of 16 requests with 16-node trees, early in their generation
        dict(name="commit_16", op="commit", B=16, Hkv=8, d=128, nodes=16, tree="chains", lo=0, hi=192, fused=True, mix=3),
        # the accepted paths of a large batch with trees of mixed sizes
        dict(name="commit_128", op="commit", B=128, Hkv=8, d=128, nodes=64, tree="random", lo=1, hi=511, fused=False, mix=4),
        # a whole cache read back (moved to a layer that wants bf16)
        dict(name="read_all", op="read", B=16, Hkv=8, d=128, lo=4096, hi=4096, start=0, fused=False, mix=5),
        # the tail of one request read back
        dict(name="read_tail", op="read", B=1, Hkv=4, d=64, lo=77, hi=77, start=1001, fused=False, mix=6),
        # one request decoding one token: latency
        dict(name="decode_one", op="attend", B=1, H=32, Hkv=8, d=128, nodes=1, tree="chains", lo=500, hi=500, window=0, sinks=0, fused=True, f32=False, mix=7),
        # 16 requests, 16-node trees, 4096 positions: the verification pass
        dict(name="tree_16x4096", op="attend", B=16, H=32, Hkv=8, d=128, nodes=16, tree="chains", lo=4096, hi=4096, window=0, sinks=0, fused=False, f32=False, mix=8),
        # a large batch decoding single tokens, ragged lengths
        dict(name="decode_64_ragged", op="attend", B=64, H=64, Hkv=8, d=128, nodes=1, tree="chains", lo=1, hi=8191, window=0, sinks=0, fused=True, f32=False, mix=9),
        # a sliding-window layer with 4 sinks over long contexts
        dict(name="tree_window", op="attend", B=32, H=16, Hkv=4, d=64, nodes=64, tree="random", lo=300, hi=32767, window=1024, sinks=4, fused=True, f32=False, mix=10),
        # best-first-sized trees of 256 nodes, single-precision output
        dict(name="trees_256", op="attend", B=8, H=32, Hkv=8, d=128, nodes=256, tree="random", lo=1500, hi=2500, window=0, sinks=0, fused=False, f32=True, mix=11),
        # one long context split over the whole GPU
        dict(name="tree_long", op="attend", B=1, H=32, Hkv=8, d=128, nodes=16, tree="chains", lo=131072, hi=131072, window=0, sinks=0, fused=False, f32=True, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "commit", "read", "attend", "attend", "attend"])
    d, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    c = dict(op=op, Hkv=Hkv, d=d, fused=rng.random() < 0.5, mix=rng.randrange(1 << 30))
    if op in ("write", "read"):
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 65536 // B))
        return dict(c, B=B, lo=max(1, hi // 3), hi=hi, start=rng.choice([0, _log(rng, 1, 900)]))
    tree = rng.choice(["chains", "random"])
    if op == "commit":
        hi = _log(rng, 1, 600)
        return dict(c, B=_log(rng, 1, 128), nodes=_log(rng, 1, 64), tree=tree, lo=hi // 4, hi=hi)
    B = _log(rng, 1, 64)
    hi = _log(rng, 16, min(65536, 262144 // B))
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    most = max(1, min(256, 8 * 2048 * 256 * 4 // (B * hi * 4)))
    return dict(c, B=B, H=Hkv * rng.choice([1, 2, 3, 4, 8]), nodes=_log(rng, 1, most), tree=tree, lo=hi // 5, hi=hi,
                window=window, sinks=rng.choice([0, 1, 4, 70]) if window else 0, f32=rng.random() < 0.5)


# ---------------------------------------------------------------- sizes and trees


def _trees(c, r):
    """Local parents of each request's tree (depth at most 16) and its accepted path."""
    parents, paths = [], []
    for b in range(c["B"]):
        n = c["nodes"] if b == 0 or c["tree"] == "chains" else int(r.integers(1, c["nodes"] + 1))
        depth = np.zeros(n, np.int64)
        p = np.full(n, -1, np.int64)
        for i in range(n):
            if c["tree"] == "chains":  # four chains from the context
                p[i] = i - 1 if i % max(1, -(-n // 4)) else -1
            elif i:
                q = int(r.integers(-1, i))
                p[i] = q if q < 0 or depth[q] < 16 else int(p[q])
            depth[i] = 1 if p[i] < 0 else depth[p[i]] + 1
        parents.append(p)
        j, path = int(r.integers(-1, n)), []
        while j >= 0:
            path.append(j)
            j = int(p[j])
        paths.append(path[::-1][:32])
    return parents, paths


def _sizes(c):
    r = np.random.default_rng(c["mix"])
    z = dict(lens=r.integers(c["lo"], c["hi"] + 1, c["B"]))
    if c["op"] in ("write", "read"):
        z["start"] = r.integers(c["start"] // 2, c["start"] + 1, c["B"]) if c["start"] else np.zeros(c["B"], np.int64)
        z["total"] = z["start"] + z["lens"]
    else:
        z["parents"], z["paths"] = _trees(c, r)
        z["total"] = z["lens"] + (32 if c["op"] == "commit" else 0)
    z["max_pages"] = max(1, int(-(-max(1, z["total"].max()) // PAGE)))
    return z


def _record(d):
    return 2 * (PAGE * d // 2 + PAGE * d // GROUP)


def work(c):
    z = _sizes(c)
    row = c["Hkv"] * c["d"] * 2 * 2  # K and V of one position in bf16
    packed = row * 17 / 64           # 4 bits and a byte for 32
    if c["op"] == "write":           # rows read and written; the whole cache read back
        n, t = int(z["lens"].sum()), int(z["total"].sum())
        return dict(bytes=n * (row + packed) + t * (row + packed), flops=0)
    if c["op"] == "read":
        return dict(bytes=int(z["lens"].sum()) * (row + packed), flops=0)
    if c["op"] == "commit":
        n, t = sum(len(p) for p in z["paths"]), int(z["lens"].sum()) + sum(len(p) for p in z["paths"])
        return dict(bytes=n * (row + packed) + t * packed + int(z["total"].sum()) * row, flops=0)
    total, flops, W, S = 0.0, 0, c["window"], c["sinks"]
    for ctx, p in zip(z["lens"].tolist(), z["parents"]):
        depth = np.zeros(len(p), np.int64)
        for i, q in enumerate(p):
            depth[i] = 1 if q < 0 else depth[q] + 1
        lo = np.maximum(0, ctx + depth - W) if W else 0 * depth
        seen = np.where(lo < ctx, ctx - lo, 0) + np.minimum(np.minimum(S, lo), ctx)
        flops += 4 * c["d"] * c["H"] * int((seen + depth).sum())
        total += int(seen.max()) * packed + len(p) * (row + c["H"] * c["d"] * (2 + (4 if c["f32"] else 2)))
    return dict(bytes=total, flops=flops)


# ---------------------------------------------------------------- the cache in torch operations


def _quantise(x):
    """[..., d] -> codes [..., d] in 1..15 and scale bytes [..., d/32] (int32)."""
    y = x.float().unflatten(-1, (-1, GROUP))
    amax = y.abs().amax(-1)
    bits = (amax / torch.full_like(amax, 7)).view(torch.int32)  # a true division: a border value has to stay one
    b = (((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - 840).clamp(0, 254)
    s = torch.ldexp((8 + b % 8).float(), b // 8 - 25).unsqueeze(-1)
    q = torch.floor(y.abs() / s + 0.5).clamp(max=7) * torch.sign(y) + 8
    return q.nan_to_num(8).to(torch.uint8).flatten(-2), torch.where(amax.isnan(), 255, b).to(torch.uint8)


def _nibbles(x):
    """[..., 16 k bytes] -> [..., 32 k elements]"""
    w = torch.stack([x & 15, x >> 4], -1).reshape(*x.shape[:-1], -1, 8)
    return w[..., NIBBLE].flatten(-2)


def _bytes(x):
    w = torch.empty_like(x).unflatten(-1, (-1, 8))
    w[..., NIBBLE] = x.unflatten(-1, (-1, 8))
    w = w.flatten(-2).unflatten(-1, (-1, 2))
    return w[..., 0] | (w[..., 1] << 4)


def _parts(cache, d):
    G = d // GROUP
    kc, ks, vc, vs = cache.split([PAGE * d // 2, PAGE * G, PAGE * d // 2, PAGE * G], -1)
    lead = cache.shape[:-1]
    return kc.reshape(*lead, G, PAGE, 16), ks.reshape(*lead, PAGE, G), vc.reshape(*lead, 2, d, 16), vs.reshape(*lead, G, PAGE)


def _unpack(cache, d):
    """records [..., record] -> K, V codes [..., 64, d] and scale bytes [..., 64, d/32]"""
    kc, ks, vc, vs = _parts(cache, d)
    k = _nibbles(kc).transpose(-2, -3).flatten(-2)
    v = _nibbles(vc).transpose(-1, -2).flatten(-3, -2)
    return k, ks, v, vs.transpose(-1, -2)


def _pack(kq, ks, vq, vs):
    k = _bytes(kq.unflatten(-1, (-1, GROUP)).transpose(-2, -3)).flatten(-3)
    v = _bytes(vq.unflatten(-2, (2, 32)).transpose(-1, -2)).flatten(-3)
    return torch.cat([k, ks.flatten(-2), v, vs.transpose(-1, -2).flatten(-2)], -1)


def _values(q, b):
    b = b.int()
    s = torch.ldexp((8 + b % 8).float(), b // 8 - 25).masked_fill(b == 255, math.nan)
    return ((q.float() - 8).unflatten(-1, (-1, GROUP)) * s.unsqueeze(-1)).flatten(-2)


def _store(cache, d, page, off, k, v):
    """Rows k, v [n, Hkv, d] into (page, off): the new cache."""
    kq, ks, vq, vs = _unpack(cache, d)
    for into, x in zip((kq, ks, vq, vs), (*_quantise(k), *_quantise(v))):
        into[page, :, off] = x
    return _pack(kq, ks, vq, vs)


def _load(cache, d, page, off, live):
    """Values [n, Hkv, d] of (page, off); zero where not live."""
    kq, ks, vq, vs = _unpack(cache, d)
    k, v = _values(kq[page, :, off], ks[page, :, off]), _values(vq[page, :, off], vs[page, :, off])
    live = live[:, None, None]
    return torch.where(live, k, 0).bfloat16(), torch.where(live, v, 0).bfloat16()


# ---------------------------------------------------------------- states


def _dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(device="cuda", dtype=dtype)


def prepare(c, seed):
    z = _sizes(c)
    g = torch.Generator(device="cuda").manual_seed(int(seed) % (1 << 62) + 1)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    B, Hkv, d, mp = c["B"], c["Hkv"], c["d"], z["max_pages"]
    pages = B * mp + 3  # a few that no request holds
    spread = torch.exp(0.5 * rand(Hkv, d))  # keys have channels that stand out
    rows = lambda n: ((rand(n, Hkv, d) * spread).bfloat16(), (0.5 * rand(n, Hkv, d)).bfloat16())  # noqa: E731
    table = torch.randperm(pages, generator=g, device="cuda")[:B * mp].reshape(B, mp).int()
    k, v = rows(pages * PAGE)  # every page holds something, past a request's end too
    per = lambda x: x.reshape(pages, PAGE, Hkv, -1).transpose(1, 2)  # noqa: E731
    cache = _pack(*(per(x) for x in (*_quantise(k), *_quantise(v))))
    del k, v
    s = dict(c=c, z=z, table=table, pages=pages, mp=mp, cache=cache.contiguous(), status=torch.zeros(4, dtype=torch.int32, device="cuda"))

    def projected(n, H):
        """q, k, v rows: packed, or views into one fused projection."""
        q, (kr, vr) = rand(n, H, d).bfloat16(), rows(n)
        s["q_stride"], s["kv_stride"] = H * d, Hkv * d
        if c["fused"]:
            both = torch.cat([q.flatten(1), kr.flatten(1), vr.flatten(1)], 1)
            s["q_stride"] = s["kv_stride"] = both.shape[1]
            q, kr, vr = (x.unflatten(1, (-1, d)) for x in both.split([H * d, Hkv * d, Hkv * d], 1))
        s["q"], s["k"], s["v"] = q, kr, vr

    offsets = lambda n: _dev(np.concatenate([[0], np.cumsum(n)]))  # noqa: E731
    s["ctx"] = _dev(z["lens"])
    s["zero"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if c["op"] in ("write", "read"):
        s["start"], s["row_offsets"], s["total"], s["all_offsets"] = _dev(z["start"]), offsets(z["lens"]), _dev(z["total"]), offsets(z["total"])
        n = int(z["lens"].sum())
        if c["op"] == "write":
            projected(n, Hkv)
            n = int(z["total"].sum())
    else:
        s["max_nodes"] = max(len(p) for p in z["parents"])
        s["node_offsets"], s["parent"] = offsets([len(p) for p in z["parents"]]), _dev(np.concatenate(z["parents"]))
        n = sum(len(p) for p in z["parents"])
        projected(n, c.get("H", Hkv))
        if c["op"] == "commit":
            s["path"], s["accept_len"] = _dev([p + [-1] * (32 - len(p)) for p in z["paths"]]), _dev([len(p) for p in z["paths"]])
            s["new_len"], s["all_offsets"] = torch.zeros_like(s["ctx"]), offsets(z["total"])
            n = int(z["total"].sum())
    if c["op"] == "attend":
        s["out"] = torch.empty(n, c["H"], d, dtype=torch.float32 if c["f32"] else torch.bfloat16, device="cuda")
        s["scale"] = 1.0 / math.sqrt(d)
    else:
        s["rows"] = n
        s["k_out"], s["v_out"] = (torch.empty(n, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if own:
        import tree_speculative_verify_tv_gb300 as tv
        s["tv"] = tv
        if c["op"] == "attend":
            need = tv.tv_qcache_attention_workspace_bytes(B, n, s["max_nodes"], c["H"], Hkv, d, mp)
            s["ws"], s["ws_bytes"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"), need
    return s


def _places(s, offsets, start, n):
    """Page, place in the page and position of each of n packed rows."""
    row = torch.arange(n, device="cuda")
    b = torch.searchsorted(offsets[1:].contiguous(), row.int(), right=True)
    pos = (start[b] + row - offsets[b]).long()
    return s["table"][b, pos // PAGE].long(), pos % PAGE, pos, b


def run(s):
    c = s["c"]
    return (_run_own if own else _run_plain)[c["op"]](s)


# ---------------------------------------------------------------- plain forms


def _plain_write(s):
    page, off, _, _ = _places(s, s["row_offsets"], s["start"], s["k"].shape[0])
    cache = _store(s["cache"], s["c"]["d"], page, off, s["k"], s["v"])
    page, off, pos, b = _places(s, s["all_offsets"], s["zero"], s["rows"])
    return _load(cache, s["c"]["d"], page, off, pos < s["total"][b])


def _plain_read(s):
    page, off, pos, b = _places(s, s["row_offsets"], s["start"], s["rows"])
    return _load(s["cache"], s["c"]["d"], page, off, pos < s["total"][b])


def _plain_commit(s):
    new_len = s["ctx"] + s["accept_len"]
    b, m = torch.nonzero(s["path"] >= 0, as_tuple=True)
    node = (s["node_offsets"][b] + s["path"][b, m]).long()
    pos = (s["ctx"][b] + m).long()
    cache = _store(s["cache"], s["c"]["d"], s["table"][b, pos // PAGE].long(), pos % PAGE, s["k"][node], s["v"][node])
    page, off, pos, b = _places(s, s["all_offsets"], s["zero"], s["rows"])
    return (new_len, *_load(cache, s["c"]["d"], page, off, pos < new_len[b]))


def _plain_attend(s):
    c, N = s["c"], s["max_nodes"]
    Hkv, d, W, S = c["Hkv"], c["d"], c["window"], c["sinks"]
    kq, ks, vq, vs = _unpack(s["cache"][s["table"].long()], d)  # [B, pages, Hkv, 64, ...]
    heads_first = lambda x: x.transpose(1, 2).flatten(2, 3)  # noqa: E731
    K, V = heads_first(_values(kq, ks)), heads_first(_values(vq, vs))
    idx = s["node_offsets"][:-1, None] + torch.arange(N, device="cuda")
    live = idx < s["node_offsets"][1:, None]
    idx = torch.where(live, idx, 0).long()
    parent = torch.where(live, s["parent"][idx], -1)
    reach = (parent[..., None] == torch.arange(N, device="cuda")) | torch.eye(N, dtype=torch.bool, device="cuda")
    for _ in range(5):  # paths of up to 32 nodes
        reach = (reach.float() @ reach.float()) > 0
    depth = reach.sum(-1)
    ctx = s["ctx"][:, None].long()
    j = torch.arange(K.shape[2], device="cuda")
    seen = (j < ctx)[:, None, :].expand(-1, N, -1)
    if W:
        at = ctx + depth - 1
        seen = seen & ((j > at[..., None] - W) | (j < S))
        reach = reach & ((depth[:, :, None] - depth[:, None, :] < W) | (at < S)[:, None, :])
    q = s["q"][idx].float().unflatten(2, (Hkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hkv, g N, d]
    kt, vt = (x[idx].float().transpose(1, 2) for x in (s["k"], s["v"]))
    g = c["H"] // Hkv
    sc = torch.cat([q @ K.transpose(2, 3), q @ kt.transpose(2, 3)], -1) * s["scale"]
    mask = torch.cat([seen, reach], -1)[:, None, None].expand(-1, Hkv, g, -1, -1).flatten(2, 3)
    sc = sc.masked_fill_(~mask, -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    l = p.sum(-1, keepdim=True)
    o = (p[..., :K.shape[2]] @ V + p[..., K.shape[2]:] @ vt) / l
    o = o.unflatten(2, (g, N)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, N, H, d]
    return o[live].to(s["out"].dtype)


_run_plain = dict(write=_plain_write, read=_plain_read, commit=_plain_commit, attend=_plain_attend)


# ---------------------------------------------------------------- the library's calls


def _own_write(s):
    c, tv = s["c"], s["tv"]
    tv.tv_qcache_write(c["B"], s["k"].shape[0], c["Hkv"], c["d"], s["pages"], s["mp"], s["row_offsets"], s["start"], s["table"],
                       s["k"], s["v"], s["kv_stride"], s["cache"], s["status"])
    tv.tv_qcache_read(c["B"], s["rows"], c["Hkv"], c["d"], s["pages"], s["mp"], s["all_offsets"], s["zero"], s["total"], s["table"],
                      s["cache"], s["k_out"], s["v_out"], c["Hkv"] * c["d"], s["status"])
    return s["k_out"], s["v_out"]


def _own_read(s):
    c = s["c"]
    s["tv"].tv_qcache_read(c["B"], s["rows"], c["Hkv"], c["d"], s["pages"], s["mp"], s["row_offsets"], s["start"], s["total"],
                           s["table"], s["cache"], s["k_out"], s["v_out"], c["Hkv"] * c["d"], s["status"])
    return s["k_out"], s["v_out"]


def _own_commit(s):
    c, tv = s["c"], s["tv"]
    tv.tv_qcache_commit(c["B"], s["k"].shape[0], s["max_nodes"], 32, c["Hkv"], c["d"], s["pages"], s["mp"], s["node_offsets"],
                        s["path"], s["accept_len"], s["ctx"], s["table"], s["k"], s["v"], s["kv_stride"], s["cache"],
                        s["new_len"], s["status"])
    tv.tv_qcache_read(c["B"], s["rows"], c["Hkv"], c["d"], s["pages"], s["mp"], s["all_offsets"], s["zero"], s["new_len"], s["table"],
                      s["cache"], s["k_out"], s["v_out"], c["Hkv"] * c["d"], s["status"])
    return s["new_len"], s["k_out"], s["v_out"]


def _own_attend(s):
    c, tv = s["c"], s["tv"]
    tv.tv_qcache_attention(c["B"], s["k"].shape[0], s["max_nodes"], c["H"], c["Hkv"], c["d"], s["pages"], s["mp"], s["node_offsets"],
                           s["parent"], s["ctx"], s["table"], c["window"], c["sinks"], s["q"], s["q_stride"], s["cache"],
                           s["k"], s["v"], s["kv_stride"], s["scale"], tv.TV_F32 if c["f32"] else tv.TV_BF16, s["out"],
                           s["ws"], s["ws_bytes"], s["status"])
    return s["out"]


_run_own = dict(write=_own_write, read=_own_read, commit=_own_commit, attend=_own_attend)


# ---------------------------------------------------------------- the definition, in 64 bits


def _exact_round(x):
    """What the cache holds for rows [n, Hkv, d], from the definition: double precision, steps by frexp."""
    y = x.double().reshape(*x.shape[:-1], -1, GROUP)
    most = y.abs().max(-1).values
    m, e = torch.frexp(most / torch.full_like(most, 7))  # m in [0.5, 1)
    m = torch.round(m * 16)                         # four significant bits, ties to even
    step = m * torch.pow(2.0, e.double() - 4)
    step = torch.clamp(step, 2.0 ** -22, 1.75 * 2.0 ** 9).unsqueeze(-1)
    t = torch.abs(y) / step
    low = torch.trunc(t)
    n = torch.minimum(low + (t - low >= 0.5).double(), torch.full_like(t, 7))
    return (torch.where(y < 0, -n, n) * step).reshape(x.shape)


def _exact_half(rec, d, value):
    """K (value False) or V of records [n, record] as doubles [n, 64, d]."""
    G = d // GROUP
    base = (PAGE * d // 2 + PAGE * G) if value else 0
    codes, scales = rec[:, base:base + PAGE * d // 2].long(), rec[:, base + PAGE * d // 2:base + PAGE * d // 2 + PAGE * G].double()
    e = torch.arange(32, device=rec.device)
    nib = (e % 8) // 2 + 4 * (e % 2)
    byte, shift = (e // 8) * 4 + nib // 2, 4 * (nib % 2)
    lines = codes.reshape(len(rec), -1, 16)
    el = ((lines[:, :, byte] >> shift) % 16 - 8).double()  # [n, lines, 32]
    size = (1 + torch.remainder(scales, 8) / 8) * torch.pow(2.0, torch.floor(scales / 8) - 22)
    if value:  # lines: (half, channel)
        el = el.reshape(len(rec), 2, d, 32).permute(0, 1, 3, 2).reshape(len(rec), PAGE, d)
        size = size.reshape(len(rec), G, PAGE).transpose(1, 2)
    else:      # lines: (group, position)
        el = el.reshape(len(rec), G, PAGE, 32).permute(0, 2, 1, 3).reshape(len(rec), PAGE, d)
        size = size.reshape(len(rec), PAGE, G)
    return el * size.repeat_interleave(GROUP, -1)


def exact(c, seed):
    s = prepare(c, seed)
    z, d, Hkv, cache = s["z"], c["d"], c["Hkv"], s["cache"]
    held = []  # per request: K, V as doubles [Hkv, positions, d]
    for b in range(c["B"]):
        rec = cache[s["table"][b].long()].transpose(0, 1).reshape(-1, cache.shape[-1])
        n = int(z["total"][b])
        half = lambda value: _exact_half(rec, d, value).reshape(Hkv, -1, d)[:, :n]  # noqa: E731
        held.append((half(False), half(True)) if c["op"] != "attend" else rec)
    if c["op"] == "attend":
        return _exact_attend(c, s, held)
    if c["op"] == "read":
        pick = [[x[:, int(a):] for x in kv] for kv, a in zip(held, z["start"])]
        return tuple(torch.cat([kv[i].transpose(0, 1) for kv in pick]) for i in (0, 1))
    new, at = [_exact_round(s["k"]), _exact_round(s["v"])], 0
    for b in range(c["B"]):
        if c["op"] == "write":
            first, n = int(z["start"][b]), int(z["lens"][b])
            rows = list(range(at, at + n))
            at += n
        else:
            first, n = int(z["lens"][b]), len(z["paths"][b])
            rows = [at + j for j in z["paths"][b]]
            at += len(z["parents"][b])
        for i in (0, 1):
            held[b][i][:, first:first + n] = new[i][rows].transpose(0, 1)
            if c["op"] == "commit":
                held[b][i][:, first + n:] = 0
    out = tuple(torch.cat([kv[i].transpose(0, 1) for kv in held]) for i in (0, 1))
    return out if c["op"] == "write" else (None, *out)


def _exact_attend(c, s, held):
    z, d, Hkv, g = s["z"], c["d"], c["Hkv"], c["H"] // c["Hkv"]
    W, S, at, out = c["window"], c["sinks"], 0, []
    for b, p in enumerate(z["parents"]):
        n, ctx = len(p), int(z["lens"][b])
        K, V = (_exact_half(held[b], d, value).reshape(Hkv, -1, d)[:, :ctx] for value in (False, True))
        K = torch.cat([K, s["k"][at:at + n].double().transpose(0, 1)], 1)
        V = torch.cat([V, s["v"][at:at + n].double().transpose(0, 1)], 1)
        seen = np.zeros((n, ctx + n), bool)
        for i in range(n):
            path, j = [], i
            while j >= 0:
                path.append(j)
                j = int(p[j])
            path = path[::-1]
            me = ctx + len(path) - 1
            seen[i, :ctx] = True
            if W:
                seen[i, min(S, ctx):max(min(S, ctx), min(ctx, me - W + 1))] = False
            for k, node in enumerate(path):
                seen[i, ctx + node] = not W or me - (ctx + k) < W or ctx + k < S
        hide = torch.as_tensor(~seen, device="cuda")
        q = s["q"][at:at + n].double().reshape(n, Hkv, g, d)
        o = torch.empty(n, Hkv, g, d, dtype=torch.float64, device="cuda")
        for h in range(g):
            w = torch.softmax((torch.matmul(q[:, :, h].transpose(0, 1), K.transpose(1, 2)) / math.sqrt(d)).masked_fill(hide, -math.inf), -1)
            o[:, :, h] = torch.matmul(w, V).transpose(0, 1)
        out.append(o.reshape(n, -1, d))
        at += n
    return torch.cat(out)
