"""Pins of the oracle's 4-bit KV cache to facts that its own code does not give (values
by hand, exhaustive neighbours, plain softmax), and the refusals of the tv_qcache_*
calls, which are made on the host before any CUDA call."""
import numpy as np
import pytest

import oracle
import tree_speculative_verify_tv_gb300 as tv
import workloads


@pytest.fixture(scope="module")
def lib():
    tv.build()
    return tv.load()


# ---------------------------------------------------------------- the format


def test_step_and_codes_by_hand():
    x = np.zeros(32)
    x[:6] = [7.0, -7.0, 0.5, -0.5, 0.49, 3.5]
    code, byte = oracle.qcache_quantise(x)
    assert byte.tolist() == [22 * 8]                       # step 1 = (8 + 0) 2^(22 - 25)
    assert code[:6].tolist() == [15, 1, 9, 7, 8, 12]       # halves away from zero
    assert code[6:].tolist() == [8] * 26
    x[0] = 7.25                                            # 7.25 / 7 = 1.0357 -> 1 (ulp 1/8)
    assert oracle.qcache_quantise(x)[1].tolist() == [22 * 8]
    x[0] = 7 * 1.0625                                      # a tie between 1 and 1.125: even
    assert oracle.qcache_quantise(x)[1].tolist() == [22 * 8]
    x[0] = 7 * 1.1875                                      # between 1.125 and 1.25: even is 1.25
    assert oracle.qcache_quantise(x)[1].tolist() == [22 * 8 + 2]


def test_range_and_special_values():
    z = np.zeros((4, 32))
    z[1, 3], z[2, 3], z[3, 3] = 1e-30, np.inf, np.nan
    z[2, 4] = 6272.0
    code, byte = oracle.qcache_quantise(z)
    assert byte[:, 0].tolist() == [0, 0, 254, 255]
    val = oracle.qcache_values(code, byte)
    assert np.all(val[:2] == 0) and val[2, 3] == val[2, 4] == 6272 and np.isnan(val[3]).all()


def test_every_value_is_exact_in_bf16_and_the_nearest_of_its_grid():
    rng = np.random.default_rng(1)
    x = workloads.bf16_bits_to_f32(workloads.f32_to_bf16_bits(
        (rng.normal(size=(400, 64)) * np.exp(rng.normal(size=(400, 1)) * 3)).astype(np.float32)))
    code, byte = oracle.qcache_quantise(x)
    val = oracle.qcache_values(code, byte)
    f32 = val.astype(np.float32)
    assert np.array_equal(workloads.bf16_bits_to_f32(workloads.f32_to_bf16_bits(f32)), f32)
    step = np.repeat(np.ldexp((8 + byte % 8).astype(float), byte.astype(int) // 8 - 25), 32, -1)
    grid = step[..., None] * np.arange(-7, 8)
    best = np.abs(grid - x[..., None]).min(-1)
    assert np.array_equal(np.abs(val - x), best)
    inside = np.abs(x) <= 6720  # beyond, values saturate at 6272
    assert np.all(np.abs(val - x)[inside] <= (step / 2)[inside])
    assert (~inside).any() and np.all(np.abs(val[~inside]) == 6272)


@pytest.mark.parametrize("d", [64, 128])
def test_record_holds_every_row_and_leaves_the_others(d):
    rng = np.random.default_rng(d)
    bytes_ = 2 * (32 * d + 2 * d)
    rec = rng.integers(0, 255, bytes_).astype(np.uint8)
    before = oracle.qcache_get(rec, d)
    rows = rng.permutation(64)[:40]
    k, v = rng.normal(size=(2, 40, d))
    for p, kr, vr in zip(rows, k, v):
        oracle.qcache_put(rec, d, int(p), kr, vr)
    K, V = oracle.qcache_get(rec, d)
    assert np.array_equal(K[rows], oracle.qcache_values(*oracle.qcache_quantise(k)))
    assert np.array_equal(V[rows], oracle.qcache_values(*oracle.qcache_quantise(v)))
    rest = np.setdiff1d(np.arange(64), rows)
    assert np.array_equal(K[rest], before[0][rest]) and np.array_equal(V[rest], before[1][rest])


def test_cache_bytes_is_seventeen_sixty_fourths_of_bf16(lib):
    for d in (64, 128):
        assert tv.tv_qcache_bytes(1, 1, d) * 64 == 2 * 2 * 64 * d * 17
        assert tv.tv_qcache_bytes(70000, 8, d) == 70000 * 8 * tv.tv_qcache_bytes(1, 1, d)
    assert tv.tv_qcache_bytes(0, 1, 128) == tv.tv_qcache_bytes(1, 0, 128) == 0
    assert tv.tv_qcache_bytes(1, 1, 96) == 0


# ---------------------------------------------------------------- windowed attention


def _attn(seed, sizes=(7, 12), ctx=(9, 30)):
    b = workloads.random_batch(np.random.default_rng(seed), list(sizes), 1, 16, 16, depth_cap=6,
                               max_depth=8)
    a = workloads.attention_inputs(b, 4, 2, 64, list(ctx), seed=seed)
    return b, a


def test_without_window_it_is_tree_attention():
    b, a = _attn(3)
    args = (b.node_offsets, b.parent, a["q_f32"], a["k_cache_f32"], a["v_cache_f32"], a["ctx_len"],
            a["k_tree_f32"], a["v_tree_f32"], a["scale"])
    want = oracle.tree_attention(*args)
    for kw in (dict(), dict(window=64), dict(window=1, sinks=64)):
        np.testing.assert_allclose(oracle.qcache_attention(*args, **kw), want, rtol=1e-12,
                                   atol=1e-13)


def test_window_of_one_returns_the_nodes_own_value():
    b, a = _attn(4)
    out = oracle.qcache_attention(b.node_offsets, b.parent, a["q_f32"], a["k_cache_f32"],
                                  a["v_cache_f32"], a["ctx_len"], a["k_tree_f32"],
                                  a["v_tree_f32"], a["scale"], window=1)
    np.testing.assert_allclose(out, np.repeat(a["v_tree_f32"], 2, axis=1), rtol=1e-12)


def test_chain_is_banded_causal_attention_with_sinks():
    torch = pytest.importorskip("torch")
    n, L, W, S = 9, 14, 6, 2
    b, a = _attn(5, sizes=(n,), ctx=(L,))
    b.parent[:] = np.arange(-1, n - 1, dtype=np.int32)
    out = oracle.qcache_attention(b.node_offsets, b.parent, a["q_f32"], a["k_cache_f32"],
                                  a["v_cache_f32"], a["ctx_len"], a["k_tree_f32"],
                                  a["v_tree_f32"], a["scale"], window=W, sinks=S)
    i, j = np.meshgrid(L + np.arange(n), np.arange(L + n), indexing="ij")
    mask = torch.from_numpy(((j <= i) & (i - j < W)) | (j < S))
    for h in range(4):
        K = np.concatenate([a["k_cache_f32"][0, h // 2, :L], a["k_tree_f32"][:, h // 2]])
        V = np.concatenate([a["v_cache_f32"][0, h // 2, :L], a["v_tree_f32"][:, h // 2]])
        t = lambda x: torch.from_numpy(x.astype(np.float64))[None, None]  # noqa: E731
        want = torch.nn.functional.scaled_dot_product_attention(
            t(a["q_f32"][:, h]), t(K), t(V), attn_mask=mask, scale=a["scale"])[0, 0]
        np.testing.assert_allclose(out[:, h], want.numpy(), rtol=1e-12, atol=1e-13)


# ---------------------------------------------------------------- refusals

A = 0x10000
P = [A + 0x1000 * i for i in range(16)]


def rows_rc(fn, **kw):
    a = dict(B=2, R=5, Hkv=2, d=128, pages=9, mp=4, offs=P[0], start=P[1], len=P[2], table=P[3],
             k=P[4], v=P[5], stride=256, cache=P[6], st=P[7])
    a.update(kw)
    if fn == "write":
        return tv.tv_qcache_write(a["B"], a["R"], a["Hkv"], a["d"], a["pages"], a["mp"], a["offs"],
                                  a["start"], a["table"], a["k"], a["v"], a["stride"], a["cache"],
                                  a["st"], stream=0, check=False)
    return tv.tv_qcache_read(a["B"], a["R"], a["Hkv"], a["d"], a["pages"], a["mp"], a["offs"],
                             a["start"], a["len"], a["table"], a["cache"], a["k"], a["v"],
                             a["stride"], a["st"], stream=0, check=False)


@pytest.mark.parametrize("fn", ["write", "read"])
@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), tv.TV_ERR_SHAPE), (dict(R=-1), tv.TV_ERR_SHAPE), (dict(Hkv=0), tv.TV_ERR_SHAPE),
    (dict(d=0), tv.TV_ERR_SHAPE), (dict(d=96), tv.TV_ERR_UNSUPPORTED),
    (dict(d=256), tv.TV_ERR_UNSUPPORTED), (dict(pages=0), tv.TV_ERR_SHAPE),
    (dict(mp=0), tv.TV_ERR_SHAPE), (dict(mp=1 << 25), tv.TV_ERR_UNSUPPORTED),
    (dict(stride=255), tv.TV_ERR_SHAPE), (dict(stride=260), tv.TV_ERR_SHAPE),
    (dict(stride=-256), tv.TV_ERR_SHAPE), (dict(R=1 << 30, Hkv=1 << 20, stride=1 << 27),
                                           tv.TV_ERR_UNSUPPORTED),
    (dict(offs=None), tv.TV_ERR_NULL), (dict(start=None), tv.TV_ERR_NULL),
    (dict(table=None), tv.TV_ERR_NULL), (dict(k=None), tv.TV_ERR_NULL),
    (dict(v=None), tv.TV_ERR_NULL), (dict(cache=None), tv.TV_ERR_NULL),
    (dict(st=None), tv.TV_ERR_NULL), (dict(st=None, B=0), tv.TV_ERR_NULL),
    (dict(offs=A + 4), tv.TV_ERR_ALIGN), (dict(k=A + 2), tv.TV_ERR_ALIGN),
    (dict(v=A + 8), tv.TV_ERR_ALIGN), (dict(cache=A + 8), tv.TV_ERR_ALIGN),
    (dict(table=A + 4), tv.TV_ERR_ALIGN), (dict(B=0), tv.TV_OK), (dict(R=0), tv.TV_OK),
])
def test_rows_calls_reject_bad_arguments(lib, fn, kw, code):
    assert rows_rc(fn, **kw) == code
    assert rows_rc("read", len=None) == tv.TV_ERR_NULL


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), tv.TV_ERR_SHAPE), (dict(T=9), tv.TV_ERR_SHAPE), (dict(mn=0), tv.TV_ERR_SHAPE),
    (dict(md=0), tv.TV_ERR_SHAPE), (dict(mn=300), tv.TV_ERR_UNSUPPORTED),
    (dict(md=33), tv.TV_ERR_UNSUPPORTED), (dict(d=32), tv.TV_ERR_UNSUPPORTED),
    (dict(stride=128), tv.TV_ERR_SHAPE), (dict(path=None), tv.TV_ERR_NULL),
    (dict(ln=None), tv.TV_ERR_NULL), (dict(ctx=None), tv.TV_ERR_NULL),
    (dict(new=None), tv.TV_ERR_NULL), (dict(k=None), tv.TV_ERR_NULL),
    (dict(st=None), tv.TV_ERR_NULL), (dict(v=A + 2), tv.TV_ERR_ALIGN),
    (dict(new=A + 4), tv.TV_ERR_ALIGN), (dict(B=0, T=0), tv.TV_OK),
])
def test_commit_rejects_bad_arguments(lib, kw, code):
    a = dict(B=2, T=5, mn=4, md=3, Hkv=2, d=128, pages=9, mp=4, offs=P[0], path=P[1], ln=P[2],
             ctx=P[3], table=P[4], k=P[5], v=P[6], stride=256, cache=P[7], new=P[8], st=P[9])
    a.update(kw)
    assert tv.tv_qcache_commit(a["B"], a["T"], a["mn"], a["md"], a["Hkv"], a["d"], a["pages"],
                               a["mp"], a["offs"], a["path"], a["ln"], a["ctx"], a["table"],
                               a["k"], a["v"], a["stride"], a["cache"], a["new"], a["st"],
                               stream=0, check=False) == code


def attn_rc(**kw):
    a = dict(B=2, T=5, mn=4, H=4, Hkv=2, d=128, pages=9, mp=4, offs=P[0], par=P[1], ctx=P[2],
             table=P[3], W=0, S=0, q=P[4], qs=512, cache=P[5], k=P[6], v=P[7], ks=256, scale=0.1,
             dt=tv.TV_F32, out=P[8], ws=P[9], wsb=1 << 40, st=P[10])
    a.update(kw)
    return tv.tv_qcache_attention(a["B"], a["T"], a["mn"], a["H"], a["Hkv"], a["d"], a["pages"],
                                  a["mp"], a["offs"], a["par"], a["ctx"], a["table"], a["W"],
                                  a["S"], a["q"], a["qs"], a["cache"], a["k"], a["v"], a["ks"],
                                  a["scale"], a["dt"], a["out"], a["ws"], a["wsb"], a["st"],
                                  stream=0, check=False)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), tv.TV_ERR_SHAPE), (dict(T=-1), tv.TV_ERR_SHAPE), (dict(T=9), tv.TV_ERR_SHAPE),
    (dict(H=3), tv.TV_ERR_SHAPE), (dict(H=0), tv.TV_ERR_SHAPE), (dict(Hkv=0), tv.TV_ERR_SHAPE),
    (dict(mn=0), tv.TV_ERR_SHAPE), (dict(mp=0), tv.TV_ERR_SHAPE), (dict(pages=0), tv.TV_ERR_SHAPE),
    (dict(d=80), tv.TV_ERR_UNSUPPORTED), (dict(mn=257), tv.TV_ERR_UNSUPPORTED),
    (dict(H=258, qs=258 * 128), tv.TV_ERR_UNSUPPORTED), (dict(W=-1), tv.TV_ERR_SHAPE),
    (dict(S=-1), tv.TV_ERR_SHAPE), (dict(qs=256), tv.TV_ERR_SHAPE), (dict(ks=258), tv.TV_ERR_SHAPE),
    (dict(scale=0.0), tv.TV_ERR_SHAPE), (dict(scale=float("nan")), tv.TV_ERR_SHAPE),
    (dict(scale=float("inf")), tv.TV_ERR_SHAPE), (dict(dt=2), tv.TV_ERR_DTYPE),
    (dict(offs=None), tv.TV_ERR_NULL), (dict(par=None), tv.TV_ERR_NULL),
    (dict(ctx=None), tv.TV_ERR_NULL), (dict(table=None), tv.TV_ERR_NULL),
    (dict(q=None), tv.TV_ERR_NULL), (dict(cache=None), tv.TV_ERR_NULL),
    (dict(k=None), tv.TV_ERR_NULL), (dict(v=None), tv.TV_ERR_NULL), (dict(out=None), tv.TV_ERR_NULL),
    (dict(st=None), tv.TV_ERR_NULL), (dict(q=A + 2), tv.TV_ERR_ALIGN),
    (dict(out=A + 4), tv.TV_ERR_ALIGN), (dict(cache=A + 8), tv.TV_ERR_ALIGN),
    (dict(mp=1 << 25), tv.TV_ERR_UNSUPPORTED), (dict(B=0, T=0), tv.TV_OK), (dict(T=0), tv.TV_OK),
])
def test_attention_rejects_bad_arguments(lib, kw, code):
    assert attn_rc(**kw) == code


def test_attention_workspace_is_checked(lib):
    need = tv.tv_qcache_attention_workspace_bytes(2, 5, 4, 4, 2, 128, 4)
    assert tv.tv_qcache_attention_workspace_bytes(2, 5, 4, 4, 2, 96, 4) == 0
    assert tv.tv_qcache_attention_workspace_bytes(0, 0, 4, 4, 2, 128, 4) == 0
    if need:
        assert attn_rc(ws=None) == tv.TV_ERR_NULL
        assert attn_rc(ws=A + 8) == tv.TV_ERR_ALIGN
        assert attn_rc(wsb=need - 1) == tv.TV_ERR_SHAPE
