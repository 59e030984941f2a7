"""Operators around the tree's verification, as cases that can be timed and compared: prompts
and single tokens through the gated linear recurrence, norms and position rotation of
queries and keys, log probabilities of tokens.

Each case is one call.  `run` computes it in elementary torch operations, or, where `own`
is set, through the library.

    prefill   H_t = e^{g_t} H_{t-1} + k_t v_t^T, o_t = H_t^T q_t for every row of ragged prompts
    decode    the same for one token of every request
    rope      x_c w_c / sqrt(mean x^2 + eps) per head, then pairs of channels rotated by
              position * frequency
    logprobs  log softmax(s x) at a token, its entropy, and the largest entries of the row
"""
import math

import numpy as np
import torch

own = False

CHUNK = 128  # tokens that the plain form of a prompt takes at once


def listed():
    return [
        # a batch of prompts through a Mamba-2-like layer
        dict(name="prefill_prompts", op="prefill", B=16, lo=4096, hi=4096, H=24, dk=128, dv=64, f32=False, out32=False, gates="token", fresh=True, fused=False, mix=1),
        # ragged prompts, rows out of a fused projection, single-precision outputs, states continued
        dict(name="prefill_ragged", op="prefill", B=12, lo=1, hi=3000, H=32, dk=128, dv=128, f32=False, out32=True, gates="token", fresh=False, fused=True, mix=2),
        # one long document, a fixed decay for each head
        dict(name="prefill_long", op="prefill", B=1, lo=32768, hi=32768, H=32, dk=128, dv=128, f32=False, out32=False, gates="head", fresh=True, fused=False, mix=3),
        # a few short chunks of prompts between decoding steps: latency
        dict(name="prefill_chunk", op="prefill", B=4, lo=30, hi=200, H=24, dk=128, dv=64, f32=False, out32=False, gates="token", fresh=False, fused=True, mix=4),
        # a large batch decoding
        dict(name="decode_128", op="decode", B=128, H=32, dk=128, dv=128, f32=False, out32=True, gates="token", fused=True, mix=5),
        # one request decoding: latency
        dict(name="decode_1", op="decode", B=1, H=24, dk=128, dv=64, f32=False, out32=False, gates="token", fused=True, mix=6),
        # prompts ahead of the cache's write
        dict(name="rope_prompts", op="rope", B=8, lo=4096, hi=4096, at=0, H=32, Hkv=8, d=128, rot=128, pairs=False, trees=False, f32=False, fused=True, mix=7),
        # 16-node trees of 16 requests, far into their contexts: latency
        dict(name="rope_trees", op="rope", B=16, lo=16, hi=16, at=100000, H=32, Hkv=8, d=128, rot=128, pairs=False, trees=True, f32=False, fused=True, mix=8),
        # ragged chunks of a single-precision model that rotates half the channels, in neighbouring pairs
        dict(name="rope_partial_f32", op="rope", B=37, lo=1, hi=500, at=3000, H=12, Hkv=12, d=64, rot=32, pairs=True, trees=False, f32=True, fused=False, mix=9),
        # the drafts' log probabilities under the target, trees of 16 requests
        dict(name="logprobs_trees", op="logprobs", R=256, N=272, V=32000, f32=False, scale=1.0, top=5, gather=True, masked=0.0, mix=10),
        # a prompt's log probabilities (scoring a document)
        dict(name="logprobs_prompt", op="logprobs", R=4096, N=4096, V=131072, f32=False, scale=1.0, top=8, gather=False, masked=0.0, mix=11),
        # one token of a grammar-masked row at a temperature: latency, odd vocabulary
        dict(name="logprobs_one", op="logprobs", R=1, N=1, V=50001, f32=True, scale=1.25, top=20, gather=False, masked=0.3, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "decode", "rope", "rope", "logprobs", "logprobs"])
    c = dict(op=op, f32=rng.random() < 0.2, mix=rng.randrange(1 << 30))
    if op in ("prefill", "decode"):
        c.update(H=rng.choice([1, 5, 8, 16, 24, 32]), dk=rng.choice([64, 128]), dv=rng.choice([64, 128]),
                 out32=rng.random() < 0.4, gates=rng.choice(["token", "token", "head"]), fused=rng.random() < 0.5)
    if op == "prefill":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, min(32768, (200000 if c["f32"] else 1000000) // (c["H"] * B))))
        return dict(c, B=B, lo=rng.choice([hi, max(1, hi // 7)]), hi=hi, fresh=rng.random() < 0.5)
    if op == "decode":
        return dict(c, B=_log(rng, 1, 128))
    if op == "rope":
        B, d, Hkv = _log(rng, 1, 64), rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
        trees = rng.random() < 0.4
        hi = _log(rng, 1, 128 if trees else max(1, 32768 // B))
        return dict(c, B=B, lo=max(1, hi // 3), hi=hi, at=_log(rng, 1, 200000), H=Hkv * rng.choice([1, 2, 4]), Hkv=Hkv, d=d,
                    rot=rng.choice([d, d, d // 2]), pairs=rng.random() < 0.4, trees=trees, fused=rng.random() < 0.5)
    V = rng.choice([32000, 50001, 131072, _log(rng, 100, 131072)])
    R = _log(rng, 1, max(1, min(4096, (1 << 27) // V)))
    return dict(c, R=R, N=R + rng.choice([0, 7]), V=V, scale=rng.choice([1.0, 1.0, 1.25, 0.7]), top=rng.choice([1, 5, 8, 20]),
                gather=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.3]))


# ---------------------------------------------------------------- sizes


def _sizes(c):
    return np.random.default_rng(c["mix"]).integers(c["lo"], c["hi"] + 1, c["B"])


def work(c):
    e, op = 4 if c["f32"] else 2, c["op"]
    if op in ("prefill", "decode"):
        n = int(_sizes(c).sum()) if op == "prefill" else c["B"]
        state = c["B"] * c["H"] * c["dk"] * c["dv"] * 4
        gates = c["H"] * 4 * (1 if c["gates"] == "head" else n)
        row = c["H"] * (e * (2 * c["dk"] + c["dv"]) + (4 if c["out32"] else 2) * c["dv"])
        return dict(bytes=n * row + gates + state * (1 if c.get("fresh") else 2), flops=4 * n * c["H"] * c["dk"] * c["dv"])
    if op == "rope":
        n = int(_sizes(c).sum())
        return dict(bytes=2 * n * (c["H"] + c["Hkv"]) * c["d"] * e, flops=10 * n * (c["H"] + c["Hkv"]) * c["d"])
    return dict(bytes=c["R"] * (c["V"] * e + 16 + 8 * c["top"]), flops=5 * c["R"] * c["V"])


# ---------------------------------------------------------------- states


def _dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(device="cuda", dtype=dtype)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) % (1 << 62) + 1)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    dtype = torch.float32 if c["f32"] else torch.bfloat16
    s = dict(c=c, status=torch.zeros(4, dtype=torch.int32, device="cuda"))

    def projected(n, **heads):
        """Rows [n, heads, width] of several projections: packed, or views into one fused projection."""
        parts = {x: (rand(n, h, d) * scale).to(dtype) for x, (h, d, scale) in heads.items()}
        if c["fused"]:
            both = torch.cat([x.flatten(1) for x in parts.values()], 1)
            cuts = both.split([x[0].numel() for x in parts.values()] if n else [0] * len(parts), 1)
            parts = {name: y.unflatten(1, x.shape[1:]) for (name, x), y in zip(parts.items(), cuts)}
        s.update(parts)
        s["stride"] = {x: y.stride(0) for x, y in parts.items()}

    if c["op"] in ("prefill", "decode"):
        B, H, dk, dv = c["B"], c["H"], c["dk"], c["dv"]
        lens = _sizes(c) if c["op"] == "prefill" else np.ones(B, np.int64)
        n = int(lens.sum())
        projected(n, q=(H, dk, 1 / math.sqrt(dk)), k=(H, dk, 1 / math.sqrt(dk)), v=(H, dv, 1.0))
        if c["gates"] == "head":  # decays from 1 - 2^-5 to 1 - 2^-10, as the heads go
            s["g"], s["g_stride"] = torch.log1p(-torch.exp2(torch.linspace(-5, -10, H, device="cuda"))), 0
        else:
            s["g"], s["g_stride"] = -torch.nn.functional.softplus(0.5 * rand(n, H) - 1), H
        fresh = c.get("fresh", False)
        s["H0"] = None if fresh else 0.05 * rand(B, H, dk, dv)
        s["H_new"] = torch.empty(B, H, dk, dv, device="cuda")
        s["out"] = torch.empty(n, H, dv, dtype=torch.float32 if c["out32"] else torch.bfloat16, device="cuda")
        s["rows"], s["max_rows"] = n, int(lens.max())
        s["offsets"] = _dev(np.concatenate([[0], np.cumsum(lens)]))
        if own:
            import tree_speculative_verify_tv_gb300 as tv
            s["tv"], s["dt"], s["odt"] = tv, tv.TV_F32 if c["f32"] else tv.TV_BF16, tv.TV_F32 if c["out32"] else tv.TV_BF16
            if c["op"] == "prefill":
                s["ws_bytes"] = tv.tv_prefill_workspace_bytes(B, n, s["max_rows"], H, dk, dv, tv.TV_DECAY_SCALAR, s["dt"])
                s["ws"] = torch.empty(max(s["ws_bytes"], 16), dtype=torch.uint8, device="cuda")
        return s
    if c["op"] == "rope":
        r = np.random.default_rng(c["mix"] + 1)
        lens = _sizes(c)
        n = int(lens.sum())
        projected(n, q=(c["H"], c["d"], 1.0), k=(c["Hkv"], c["d"], 2.0), v=(c["Hkv"], c["d"], 1.0))
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * rand(c["d"])).to(dtype) for _ in range(2))
        s["rows"], s["offsets"] = n, _dev(np.concatenate([[0], np.cumsum(lens)]))
        s["start"] = _dev(r.integers(c["at"] // 2, c["at"] + 1, c["B"]))
        s["depth"] = None
        if c["trees"]:  # four chains below each request's context
            s["depth"] = _dev(np.concatenate([1 + np.arange(m) % max(1, -(-m // 4)) % 32 for m in lens]))
        s["freq"] = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        s["q_out"], s["k_out"] = (torch.empty(n, h, c["d"], dtype=dtype, device="cuda") for h in (c["H"], c["Hkv"]))
        if own:
            import tree_speculative_verify_tv_gb300 as tv
            s["tv"], s["dt"] = tv, tv.TV_F32 if c["f32"] else tv.TV_BF16
        return s
    R, N, V, K = c["R"], c["N"], c["V"], c["top"]
    x = 2.5 * rand(N, V)
    if c["masked"]:  # tokens that a grammar forbids
        x.masked_fill_(torch.rand(N, V, generator=g, device="cuda") < c["masked"], -math.inf)
    s["logits"] = x.to(dtype)
    s["rows"] = torch.randint(0, N, (R,), generator=g, device="cuda").int() if c["gather"] else None
    s["tokens"] = torch.randint(0, V, (R,), generator=g, device="cuda").int()
    s["logprob"], s["entropy"] = (torch.empty(R, device="cuda") for _ in range(2))
    s["top_token"], s["top_logprob"] = torch.empty(R, K, dtype=torch.int32, device="cuda"), torch.empty(R, K, device="cuda")
    if own:
        import tree_speculative_verify_tv_gb300 as tv
        s["tv"], s["dt"] = tv, tv.TV_F32 if c["f32"] else tv.TV_BF16
    return s


def run(s):
    return (_run_own if own else _run_plain)[s["c"]["op"]](s)


# ---------------------------------------------------------------- plain forms


def _plain_prefill(s):
    """Chunks of every request at once; only the states at the chunks' starts follow one another."""
    c, B, H = s["c"], s["c"]["B"], s["c"]["H"]
    n = -(-s["max_rows"] // CHUNK)
    first, end = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
    at = first + torch.arange(n * CHUNK, device="cuda")
    live = at < end
    at = torch.where(live, at, 0)

    def chunks(x):  # [rows, H, w] -> [B, H, n, CHUNK, w], zeros past a request's end
        x = torch.where(live[..., None, None], x[at].float(), 0.0)
        return x.unflatten(1, (n, CHUNK)).permute(0, 3, 1, 2, 4)

    q, k, v = chunks(s["q"]), chunks(s["k"]), chunks(s["v"])
    g = s["g"].expand(s["rows"], H) if s["g"].dim() == 1 else s["g"]
    L = chunks(g[..., None])[..., 0].double().cumsum(-1)  # decays up to each row of a chunk
    last = L[..., -1:]
    states = torch.empty(B, H, n, c["dk"], c["dv"], device="cuda")
    H_t = torch.zeros_like(states[:, :, 0]) if s["H0"] is None else s["H0"].clone()
    added = (k * torch.exp((last - L).float())[..., None]).transpose(-1, -2) @ v
    kept = torch.exp(last).float()[..., None]
    for i in range(n):
        states[:, :, i] = H_t
        H_t = kept[:, :, i] * H_t + added[:, :, i]
    d = (L[..., :, None] - L[..., None, :]).float()
    past = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    w = (q @ k.transpose(-1, -2)) * torch.exp(d.masked_fill_(~past, -math.inf))
    o = w @ v + torch.exp(L.float())[..., None] * (q @ states)
    o = o.permute(0, 2, 3, 1, 4).flatten(1, 2)
    return o[live].to(s["out"].dtype), H_t


def _plain_decode(s):
    H = s["H0"] * torch.exp(s["g"])[..., None, None] + s["k"].float()[..., :, None] * s["v"].float()[..., None, :]
    return (s["q"].float()[..., :, None] * H).sum(-2).to(s["out"].dtype), H


def _plain_rope(s):
    c, rot = s["c"], s["c"]["rot"]
    row = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["offsets"][1:].contiguous(), row.int(), right=True)
    pos = s["start"][b].long() + (row - s["offsets"][b] if s["depth"] is None else s["depth"] - 1)
    angle = pos.double()[:, None] * s["freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def one(x, weight):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
        r, rest = x[..., :rot], x[..., rot:]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["pairs"] else (r[..., :rot // 2], r[..., rot // 2:])
        a, b = a * cos - b * sin, b * cos + a * sin
        r = torch.stack([a, b], -1).flatten(-2) if c["pairs"] else torch.cat([a, b], -1)
        return torch.cat([r, rest], -1).to(s["q_out"].dtype)

    return one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])


def _plain_logprobs(s):
    c = s["c"]
    raw = s["logits"] if s["rows"] is None else s["logits"][s["rows"].long()]
    raw = raw[:c["R"]].float()
    x = raw * c["scale"]
    x = x - x.amax(-1, keepdim=True)
    p = torch.exp(x)
    z = p.sum(-1, keepdim=True)
    x = x - torch.log(z)
    entropy = -torch.where(p > 0, p * x, 0.0).sum(-1) / z[:, 0]
    token = s["tokens"].long()[:, None]
    bits = (raw + 0.0).view(torch.int32)  # as whole numbers of the same order, the lower index ahead
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() * (1 << 20) - torch.arange(c["V"], device="cuda")
    top = order.topk(c["top"], -1).indices
    return x.gather(-1, token)[:, 0], entropy, top.int(), x.gather(-1, top)


_run_plain = dict(prefill=_plain_prefill, decode=_plain_decode, rope=_plain_rope, logprobs=_plain_logprobs)


# ---------------------------------------------------------------- the library's calls


def _own_prefill(s):
    c, tv = s["c"], s["tv"]
    tv.tv_prefill(c["B"], s["rows"], s["max_rows"], c["H"], c["dk"], c["dv"], tv.TV_DECAY_SCALAR, s["dt"], s["offsets"], s["H0"],
                  s["q"], s["stride"]["q"], s["k"], s["stride"]["k"], s["v"], s["stride"]["v"], s["g"], s["g_stride"],
                  s["odt"], s["out"], s["H_new"], s["ws"], s["ws_bytes"], s["status"])
    return s["out"], s["H_new"]


def _own_decode(s):
    c, tv = s["c"], s["tv"]
    tv.tv_decode(c["B"], c["H"], c["dk"], c["dv"], tv.TV_DECAY_SCALAR, s["dt"], None, s["H0"],
                 s["q"], s["stride"]["q"], s["k"], s["stride"]["k"], s["v"], s["stride"]["v"], s["g"], s["g_stride"],
                 s["odt"], s["out"], s["H_new"])
    return s["out"], s["H_new"]


def _own_rope(s):
    c, tv = s["c"], s["tv"]
    tv.tv_qk_norm_rope(c["B"], s["rows"], c["H"], c["Hkv"], c["d"], c["rot"], tv.TV_ROPE_PAIRS if c["pairs"] else tv.TV_ROPE_HALVES,
                       s["dt"], s["offsets"], s["start"], s["depth"], s["q"], s["stride"]["q"], s["k"], s["stride"]["k"],
                       s["q_weight"], s["k_weight"], 1e-6, s["freq"], s["q_out"], c["H"] * c["d"], s["k_out"], c["Hkv"] * c["d"],
                       s["status"])
    return s["q_out"], s["k_out"]


def _own_logprobs(s):
    c, tv = s["c"], s["tv"]
    tv.tv_logprobs(c["R"], c["N"], c["V"], s["dt"], s["logits"], c["V"], s["rows"], s["tokens"], c["scale"], c["top"],
                   s["logprob"], s["entropy"], s["top_token"], s["top_logprob"], s["status"])
    return s["logprob"], s["entropy"], s["top_token"], s["top_logprob"]


_run_own = dict(prefill=_own_prefill, decode=_own_decode, rope=_own_rope, logprobs=_own_logprobs)


# ---------------------------------------------------------------- the definitions, in 64 bits


def _exact_tokens(c, s):
    """The recurrence, token after token, for all requests and heads at once."""
    offsets = s["offsets"].tolist()
    B, H = c["B"], c["H"]
    state = torch.zeros(B, H, c["dk"], c["dv"], dtype=torch.float64, device="cuda")
    if s["H0"] is not None:
        state += s["H0"]
    q, k, v = (s[x].double() for x in "qkv")
    decay = torch.exp(s["g"].double())
    out = torch.zeros(s["rows"], H, c["dv"], dtype=torch.float64, device="cuda")
    by_length = sorted(range(B), key=lambda b: offsets[b] - offsets[b + 1])  # the longest first
    lens = [offsets[b + 1] - offsets[b] for b in by_length]
    begin = torch.tensor([offsets[b] for b in by_length], device="cuda")
    state, m = state[by_length], B
    for t in range(lens[0]):
        while lens[m - 1] <= t:
            m -= 1
        at, now = begin[:m] + t, state[:m]
        now *= (decay if c["gates"] == "head" else decay[at])[..., None, None]
        torch.addcmul(now, k[at].unsqueeze(-1), v[at].unsqueeze(-2), out=now)
        out[at] = torch.matmul(q[at].unsqueeze(-2), now).squeeze(-2)
    back = torch.empty_like(state)
    back[by_length] = state
    return out, back


def _exact_rope(c, s):
    offsets, start = s["offsets"].tolist(), s["start"].tolist()
    pos = np.concatenate([start[b] + np.arange(offsets[b + 1] - offsets[b]) for b in range(c["B"])])
    if s["depth"] is not None:
        pos = np.concatenate([np.full(offsets[b + 1] - offsets[b], start[b]) for b in range(c["B"])]) + s["depth"].cpu().numpy() - 1
    half = c["rot"] // 2
    theta = np.outer(pos, [10000.0 ** (-2.0 * i / c["rot"]) for i in range(half)])
    turn = torch.as_tensor(np.exp(1j * theta), device="cuda")[:, None]
    low = torch.arange(half, device="cuda") * (2 if c["pairs"] else 1)
    high = low + (1 if c["pairs"] else half)
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.double()
        y = y / torch.sqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / c["d"] + 1e-6) * w.double()
        z = torch.complex(y[..., low], y[..., high]) * turn
        y[..., low], y[..., high] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_logprobs(c, s):
    rows = range(c["R"]) if s["rows"] is None else s["rows"].tolist()
    got = [], [], []
    for i, r in enumerate(rows):
        x = torch.log_softmax(s["logits"][r].double() * c["scale"], -1)
        best = torch.sort(s["logits"][r].double(), descending=True, stable=True).indices[:c["top"]]
        seen = x[x > -math.inf]
        for into, value in zip(got, (x[s["tokens"][i].long()], -(seen * torch.exp(seen)).sum(), x[best])):
            into.append(value)
    logprob, entropy, top = (torch.stack(x) for x in got)
    return logprob, entropy, None, top


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("prefill", "decode"):
        return _exact_tokens(c, s)
    return (_exact_rope if c["op"] == "rope" else _exact_logprobs)(c, s)
