"""Pins of the oracle's prompts, norms with rotation and log probabilities (no GPU)."""
import numpy as np
import pytest

import oracle
import workloads


@pytest.mark.parametrize("diag", [False, True])
def test_a_prompt_is_a_chain_of_draft_nodes(diag):
    """The recurrence over a prompt is the tree verification of one chain, and its state the
    commit of the whole chain."""
    rng = np.random.default_rng(1)
    n = 9
    b = workloads.assemble(rng, [np.arange(n) - 1], 2, 8, 16, decay="diag" if diag else "scalar",
                           qkv_dtype="f32", g_kind="softplus01", h0_std=0.3, max_depth=16)
    out, S = oracle.prefill([0, n], b.q, b.k, b.v, b.g, b.H0, diag)
    for h, ref in oracle.verify(b).items():
        assert np.allclose(out[:, h], ref, rtol=1e-13, atol=1e-13)
    path = np.full((1, 16), -1, np.int32)
    path[0, :n] = np.arange(n)
    for h, ref in oracle.commit(b, np.array([n], np.int32), path).items():
        assert np.allclose(S[0, h], ref, rtol=1e-13, atol=1e-13)


def test_a_prompt_without_decay_is_a_sum():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(3, 20, 2, 8))
    out, S = oracle.prefill([0, 12, 12, 20], q, k, v, np.zeros((20, 2)))
    assert np.allclose(S[0], np.einsum("thc,thd->hcd", k[:12], v[:12]))
    assert not S[1].any()
    w = np.einsum("thc,shc->hts", q[12:], k[12:]) * np.tri(8)
    assert np.allclose(out[12:], np.einsum("hts,shd->thd", w, v[12:]))


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation(pairs):
    """Rotations keep lengths, scores depend on distances only, position 0 and channels past the
    rotated ones stay."""
    rng = np.random.default_rng(3)
    x = rng.normal(size=(2, 1, 16))
    f = 100.0 ** -np.arange(6)
    rope = lambda y, p: oracle.qk_norm_rope(y, p, None, None, f, pairs)  # noqa: E731
    assert np.array_equal(rope(x, [0, 0]), x)
    y = rope(x, [5, 1000])
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1)) and np.array_equal(y[..., 12:], x[..., 12:])
    a, b = rope(x, [7, 3]), rope(x, [107, 103])
    assert np.allclose((a[0] * a[1]).sum(), (b[0] * b[1]).sum())
    one = rope(np.eye(16)[None, :1], [1])[0, 0]
    hit = 1 if pairs else 6
    assert np.isclose(one[0], np.cos(1)) and np.isclose(one[hit], np.sin(1))


def test_norm():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    y = oracle.qk_norm_rope(x, [0], np.array([1.0, 2.0, 1.0, 1.0]), 0.0, np.zeros(0), False)
    assert np.allclose(y, [[[1.2, 3.2, 0.0, 0.0]]])


def test_logprobs():
    x = np.array(
        [[np.log(0.5), np.log(0.25), np.log(0.25), -np.inf], [-np.inf] * 4, [0, np.nan, 1, np.inf]])
    lp, ent, tt, tl = oracle.logprobs(x, [0, 0, 1, 2, -1], [1, 3, 2, 0, 0], 1.0, 3)
    assert np.isclose(lp[0], np.log(0.25)) and lp[1] == -np.inf and lp[2] == -np.inf
    assert np.isnan(lp[3]) and lp[4] == 0 and ent[4] == 0 and ent[2] == 0
    assert np.isclose(ent[0], 1.5 * np.log(2))
    assert tt.tolist() == [[0, 1, 2], [0, 1, 2], [0, 1, 2], [1, 3, 2], [-1] * 3]
    assert np.allclose(tl[0], np.log([0.5, 0.25, 0.25])) and (tl[2] == -np.inf).all()
    half = oracle.logprobs(np.array([[0.0, 2.0]]), [0], [1], 0.5, 1)[0][0]
    assert np.isclose(half, -np.log1p(np.exp(-1)))
