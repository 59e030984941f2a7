"""tv_logprobs against log softmax in 64 bits; the top tokens exactly.

Bound: scaling, the difference from the maximum, the logarithm and the two differences round at
2^-24 of their values, the sum of exponentials (2^-22 each) adds at most 2^-20 to its logarithm
and, for the entropy, to sum p |ln p|; a scaled logit's rounding (2^-24 of it) moves an
exponential by as much."""
import numpy as np
import pytest

import oracle
import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()


def values(rng, shape, f32, spread=3.0):
    x = (spread * rng.normal(size=shape)).astype(np.float32)
    return x if f32 else workloads.bf16_bits_to_f32(workloads.f32_to_bf16_bits(x))


def call(x, f32, rows, tokens, scale, top, stride=None, entropy=True, status=None):
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    N, V = x.shape
    dev = torch.from_numpy(x).cuda().to(torch.float32 if f32 else torch.bfloat16)
    if stride:
        wide = torch.full((N, stride), float("nan"), dtype=dev.dtype, device="cuda")
        wide[:, :V] = dev
        dev = wide
    ints = lambda y: None if y is None else torch.from_numpy(np.asarray(y, np.int32)).cuda()  # noqa: E731
    R = len(rows) if rows is not None else len(tokens) if tokens is not None else N
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    lp = nan(R) if tokens is not None else None
    ent = nan(R) if entropy else None
    tt, tl = torch.full((R, top), -7, dtype=torch.int32, device="cuda"), nan(R, top)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tv.tv_logprobs(R, N, V, tv.TV_F32 if f32 else tv.TV_BF16, dev, stride or V, ints(rows),
                   ints(tokens), scale, top, lp, ent, tt if top else None, tl if top else None, st)
    torch.cuda.synchronize()
    if status is None:
        assert int(st[0]) == 0
    else:
        assert int(st[0]) == status
    host = lambda y: None if y is None else y.cpu().numpy()  # noqa: E731
    return host(lp), host(ent), host(tt), host(tl)


def check(x, f32, rows, tokens, scale, top, got):
    R = len(rows) if rows is not None else len(tokens) if tokens is not None else len(x)
    at = rows if rows is not None else range(R)
    want = oracle.logprobs(x, at, tokens if tokens is not None else [-1] * R, scale, top)
    seen = np.where(np.isfinite(x), np.abs(x.astype(np.float64)), 0) * scale
    size = np.array([seen[max(r, 0)].max() for r in at]) if R else np.zeros(0)
    for i, (g, w) in enumerate(zip(got, want)):
        if g is None:
            continue
        if i == 2:
            assert np.array_equal(g, w)
            continue
        g, w = g.astype(np.float64), w.astype(np.float64)
        fine = np.isfinite(w)
        assert np.array_equal(np.isnan(g), np.isnan(w))
        assert np.array_equal(g[~fine & ~np.isnan(w)], w[~fine & ~np.isnan(w)])
        s = size[:, None] if i == 3 else size
        bound = 2.0 ** -22 * (s + np.abs(np.where(fine, w, 0))) + 2.0 ** -19
        if i == 1:  # p's error (2^-24 of the scaled logits and 2^-20) on the entropy's terms
            bound = (2.0 ** -22 * s + 2.0 ** -19) * (1 + np.abs(np.where(fine, w, 0)))
        assert (np.abs(g - w) <= bound)[fine].all(), (i, float(np.abs(g - w)[fine].max()))


def run(seed, R, V, f32, top, scale=1.0, spread=3.0, stride=None):
    rng = np.random.default_rng(seed)
    x = values(rng, (R, V), f32, spread)
    tokens = rng.integers(0, V, R)
    check(x, f32, None, tokens, scale, top, call(x, f32, None, tokens, scale, top, stride))


@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 257, 1000, 4099, 32000, 50001, 131072])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("R", [1, 5])
def test_vocabularies(V, f32, R):
    run(1, R, V, f32, min(5, V))


@pytest.mark.parametrize("top", [0, 1, 2, 20, 31, 32])
@pytest.mark.parametrize("f32", [False, True])
def test_numbers_of_alternatives(top, f32):
    run(2, 9, 5003, f32, top)


@pytest.mark.parametrize("R", [200, 700])
@pytest.mark.parametrize("V", [1000, 8192])
@pytest.mark.parametrize("f32", [False, True])
def test_many_rows(R, V, f32):
    run(3, R, V, f32, 8)


@pytest.mark.parametrize("scale", [0.01, 0.7, 1.25, 100.0])
def test_scales(scale):
    run(4, 6, 3001, False, 6, scale)
    run(4, 6, 3001, True, 6, scale)


@pytest.mark.parametrize("stride", [1001, 1008, 1037])
@pytest.mark.parametrize("f32", [False, True])
def test_strides_and_alignment(stride, f32):
    run(5, 11, 1000, f32, 4, stride=stride)


def test_rows_gathered_and_padded():
    import tree_speculative_verify_tv_gb300 as tv
    rng = np.random.default_rng(6)
    x = values(rng, (7, 999), False)
    rows, tokens = [3, 3, -1, 0, 6, 6, -5], [5, -1, 4, 998, 0, 0, -2]
    check(x, False, rows, tokens, 1.0, 3, call(x, False, rows, tokens, 1.0, 3))
    got = call(x, False, [7, 2, 2], [0, 999, 5], 1.0, 2, status=tv.TV_ERR_SHAPE)
    check(x, False, [-1, 2, 2], [-1, -1, 5], 1.0, 2, got)


def test_parts_of_the_results():
    rng = np.random.default_rng(7)
    x = values(rng, (4, 777), True)
    check(x, True, None, [1, 2, 3, 4], 1.0, 0, call(x, True, None, [1, 2, 3, 4], 1.0, 0))
    check(x, True, None, None, 1.0, 3, call(x, True, None, None, 1.0, 3, entropy=False))
    check(x, True, None, None, 1.0, 0, call(x, True, None, None, 1.0, 0))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [40, 2500, 40000])
def test_ties(f32, V):
    """Few distinct values: the lower index first; all equal; rising and falling rows; a block of
    large values that one thread or warp would own."""
    rng = np.random.default_rng(8)
    x = np.stack([rng.integers(0, 3, V) * 0.5, np.zeros(V), np.arange(V) // 4 * 0.25 - V / 32,
                  -np.arange(V) // 4 * 0.25, np.where(np.arange(V) % 256 < 2, 3.0, 0.0),
                  np.where((np.arange(V) >= 8) & (np.arange(V) < 40), 2.0, -1.0),
                  np.where(np.arange(V) % 2048 < 8, np.arange(V) / 65536.0, -9.0),
                  np.where(np.arange(V) == V - 1, 5.0, -0.0)]).astype(np.float32)
    if not f32:
        x = workloads.bf16_bits_to_f32(workloads.f32_to_bf16_bits(x))
    tokens = rng.integers(0, V, len(x))
    check(x, f32, None, tokens, 1.0, 32, call(x, f32, None, tokens, 1.0, 32))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [33, 1003, 40000])
def test_masked_infinite_and_bad_rows(f32, V):
    rng = np.random.default_rng(9)
    x = values(rng, (12, V), f32)
    big = np.finfo(np.float32).max if f32 else 3.38953139e38
    x[0, rng.random(V) < 0.9] = -np.inf
    x[1] = -np.inf
    x[2, :] = -np.inf
    x[2, V // 2] = 1.0
    x[3, 5] = np.inf
    x[4, 7] = np.nan
    x[5, 3:9] = np.nan
    x[5, 20] = np.inf
    x[6] = -big                      # the type's lowest value everywhere
    x[7, 1:] = -big
    x[8, ::2] = -big
    x[9] = np.where(np.arange(V) % 2, 0.0, -0.0)
    x[10, 3], x[10, 9] = big, big    # the largest values: the others' probabilities vanish
    x[11] = 1e-30
    tokens = np.array([3, 4, V // 2, 5, 6, 2, 1, 1, 2, 0, 4, V - 1])
    check(x, f32, None, tokens, 1.0, 20, call(x, f32, None, tokens, 1.0, 20))


def test_the_first_alternative_is_the_greedy_choice():
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    b = workloads.config2(seed=31, B=4, H=1)
    rl, nl = workloads.target_logits(b, 32000, seed=3, **{})
    both = np.concatenate([rl, nl])
    x = workloads.bf16_bits_to_f32(both)
    top = call(x, False, None, None, 1.0, 1)[2][:, 0]
    assert np.array_equal(top, oracle.argmax_rows(both))


def test_rows_past_32_bits_of_offset():
    """A row that begins past 2^32 bytes (and 2^31 elements) of the logits."""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    V, N = 131072, 16500
    logits = torch.zeros((N, V), dtype=torch.bfloat16, device="cuda")
    logits[N - 1, 77] = 4.0
    lp, ent = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    tt, tl = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    row, token = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (N - 1, 78))
    tv.tv_logprobs(1, N, V, tv.TV_BF16, logits, V, row, token, 1.0, 1, lp, ent, tt, tl, st)
    z = V - 1 + np.exp(4.0)
    assert int(tt[0]) == 77 and abs(float(tl[0]) - (4 - np.log(z))) < 2.0 ** -18
    assert abs(float(lp[0]) + np.log(z)) < 2.0 ** -18 and int(st[0]) == 0


def test_the_largest_scale():
    """The base-2 factor is past single precision, the scale is not."""
    x = np.array([[0.0, 0.5, 1.0, -1.0]], np.float32)
    lp, ent, tt, tl = call(x, True, [0, 0, 0], [0, 1, 2], 2.9e38, 3)
    want = np.array([-2.9e38, -1.45e38, 0.0])
    assert np.allclose(lp, want, rtol=2.0 ** -22) and (ent == 0).all()
    assert (tt == [2, 1, 0]).all() and np.allclose(tl, want[::-1], rtol=2.0 ** -22)


def test_the_longest_row():
    """2^31 - 1 equal logits: the sum is one row's, ties go to the first indexes."""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    V = 2 ** 31 - 1
    logits = torch.zeros(V, dtype=torch.bfloat16, device="cuda")
    lp, ent = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    tt, tl = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(3, device="cuda")
    st, token = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (0, V - 1))
    tv.tv_logprobs(1, 1, V, tv.TV_BF16, logits, V, None, token, 1.0, 3, lp, ent, tt, tl, st)
    assert tt.tolist() == [0, 1, 2] and int(st[0]) == 0
    for y in (lp, -ent, tl):  # ln z: 2^-20 of the sum, and two roundings of 21.5
        assert (y.double() + np.log(V)).abs().max() <= 2.0 ** -18


def test_replayed_from_a_graph():
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    rng = np.random.default_rng(10)
    x = torch.from_numpy(values(rng, (3, 30011), True)).cuda()
    tokens = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    lp, ent = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    tt, tl = torch.empty(3, 4, dtype=torch.int32, device="cuda"), torch.empty(3, 4, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run():
        tv.tv_logprobs(3, 3, 30011, tv.TV_F32, x, 30011, None, tokens, 1.0, 4, lp, ent, tt, tl, st)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    x.copy_(torch.from_numpy(values(rng, (3, 30011), True)))
    graph.replay()
    torch.cuda.synchronize()
    check(x.cpu().numpy(), True, None, [5, 6, 7], 1.0, 4,
          [y.cpu().numpy() for y in (lp, ent, tt, tl)])
