"""Refusals of tv_prefill, tv_decode, tv_qk_norm_rope and tv_logprobs, on the host: every call
below fails (or has nothing to do) before it touches its fake addresses."""
import pytest

import tree_speculative_verify_tv_gb300 as tv

P = [0x10000 + 0x1000 * i for i in range(20)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    tv.build()
    return tv.load()


PREFILL = dict(B=2, total_rows=9, max_rows=8, H=3, dk=64, dv=64, decay=0, qkv_dtype=0,
               row_offsets=P[0], H0=P[1], q=P[2], q_stride=192, k=P[3], k_stride=192, v=P[4],
               v_stride=192, g=P[5], g_stride=3, out_dtype=0, out=P[6], H_new=P[7],
               workspace=P[8], workspace_bytes=64, dev_status=P[9])
DECODE = dict(B=2, H=3, dk=64, dv=64, decay=0, qkv_dtype=0, active=P[0], H0=P[1], q=P[2],
              q_stride=192, k=P[3], k_stride=192, v=P[4], v_stride=192, g=P[5], g_stride=3,
              out_dtype=0, out=P[6], H_new=P[7])
ROPE = dict(B=2, total_rows=9, H=4, Hkv=2, d=64, rotary_dim=64, layout=0, dtype=0,
            row_offsets=P[0], start=P[1], depth=P[2], q=P[3], q_stride=256, k=P[4], k_stride=128,
            q_weight=P[5], k_weight=P[6], eps=1e-6, inv_freq=P[7], q_out=P[8], q_out_stride=256,
            k_out=P[9], k_out_stride=128, dev_status=P[10])
LOGPROBS = dict(R=4, num_rows=4, vocab=100, logits_dtype=0, logits=P[0], row_stride=100,
                rows=P[1], tokens=P[2], scale=1.0, top_k=5, logprob=P[3], entropy=P[4],
                top_token=P[5], top_logprob=P[6], dev_status=P[7])


def rc(f, base, **kw):
    return f(**{**base, **kw}, stream=0, check=False)


RECURRENCE = [
    (dict(B=-1), tv.TV_ERR_SHAPE), (dict(H=0), tv.TV_ERR_SHAPE), (dict(dk=12), tv.TV_ERR_SHAPE),
    (dict(dv=0), tv.TV_ERR_SHAPE), (dict(dk=264, q_stride=800, k_stride=800), tv.TV_ERR_UNSUPPORTED),
    (dict(dv=264, v_stride=800), tv.TV_ERR_UNSUPPORTED), (dict(decay=2), tv.TV_ERR_DTYPE),
    (dict(qkv_dtype=3), tv.TV_ERR_DTYPE), (dict(out_dtype=2), tv.TV_ERR_DTYPE),
    (dict(q_stride=184), tv.TV_ERR_SHAPE), (dict(k_stride=196), tv.TV_ERR_SHAPE),
    (dict(v_stride=0), tv.TV_ERR_SHAPE), (dict(g_stride=2), tv.TV_ERR_SHAPE),
    (dict(g_stride=-3), tv.TV_ERR_SHAPE), (dict(decay=1, g_stride=64), tv.TV_ERR_SHAPE),
    (dict(q=None), tv.TV_ERR_NULL), (dict(k=None), tv.TV_ERR_NULL), (dict(v=None), tv.TV_ERR_NULL),
    (dict(g=None), tv.TV_ERR_NULL), (dict(out=None), tv.TV_ERR_NULL),
    (dict(H_new=None), tv.TV_ERR_NULL), (dict(q=P[2] + 8), tv.TV_ERR_ALIGN),
    (dict(g=P[2] + 2), tv.TV_ERR_ALIGN), (dict(out=P[2] + 8), tv.TV_ERR_ALIGN),
    (dict(H0=P[2] + 4), tv.TV_ERR_ALIGN), (dict(H_new=P[2] + 4), tv.TV_ERR_ALIGN),
    (dict(H=1 << 30, B=4, total_rows=0, q_stride=1 << 40, k_stride=1 << 40, v_stride=1 << 40,
          g_stride=0), tv.TV_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", RECURRENCE + [
    (dict(total_rows=-1), tv.TV_ERR_SHAPE), (dict(total_rows=17), tv.TV_ERR_SHAPE),
    (dict(max_rows=0), tv.TV_ERR_SHAPE), (dict(row_offsets=None), tv.TV_ERR_NULL),
    (dict(dev_status=None), tv.TV_ERR_NULL), (dict(row_offsets=P[0] + 4), tv.TV_ERR_ALIGN),
    (dict(workspace=P[8] + 8), tv.TV_ERR_ALIGN), (dict(B=0, total_rows=0), tv.TV_OK),
])
def test_prefill(kw, code):
    assert rc(tv.tv_prefill, PREFILL, **kw) == code


@pytest.mark.parametrize("kw,code", [(kw, code) for kw, code in RECURRENCE
                                     if "total_rows" not in kw] + [
    (dict(H0=None), tv.TV_ERR_NULL), (dict(active=P[0] + 4), tv.TV_ERR_ALIGN),
    (dict(B=0), tv.TV_OK), (dict(H=1 << 30, B=4, q_stride=1 << 40, k_stride=1 << 40,
                                 v_stride=1 << 40, g_stride=0), tv.TV_ERR_UNSUPPORTED),
])
def test_decode(kw, code):
    assert rc(tv.tv_decode, DECODE, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), tv.TV_ERR_SHAPE), (dict(total_rows=-1), tv.TV_ERR_SHAPE),
    (dict(H=0), tv.TV_ERR_SHAPE), (dict(Hkv=-1), tv.TV_ERR_SHAPE), (dict(d=0), tv.TV_ERR_SHAPE),
    (dict(d=96, q_stride=400, k_stride=400), tv.TV_ERR_UNSUPPORTED),
    (dict(rotary_dim=72), tv.TV_ERR_SHAPE), (dict(rotary_dim=-8), tv.TV_ERR_SHAPE),
    (dict(rotary_dim=20), tv.TV_ERR_SHAPE), (dict(layout=2), tv.TV_ERR_DTYPE),
    (dict(dtype=2), tv.TV_ERR_DTYPE), (dict(q_stride=248), tv.TV_ERR_SHAPE),
    (dict(q_stride=260), tv.TV_ERR_SHAPE), (dict(k_stride=120), tv.TV_ERR_SHAPE),
    (dict(q_out_stride=8), tv.TV_ERR_SHAPE), (dict(k_out_stride=132), tv.TV_ERR_SHAPE),
    (dict(eps=float("nan")), tv.TV_ERR_SHAPE), (dict(eps=float("inf")), tv.TV_ERR_SHAPE),
    (dict(eps=-float("inf")), tv.TV_ERR_SHAPE), (dict(dev_status=None), tv.TV_ERR_NULL),
    (dict(row_offsets=None), tv.TV_ERR_NULL), (dict(start=None), tv.TV_ERR_NULL),
    (dict(q=None), tv.TV_ERR_NULL), (dict(k=None), tv.TV_ERR_NULL),
    (dict(q_out=None), tv.TV_ERR_NULL), (dict(k_out=None), tv.TV_ERR_NULL),
    (dict(inv_freq=None), tv.TV_ERR_NULL), (dict(q=P[3] + 2), tv.TV_ERR_ALIGN),
    (dict(depth=P[3] + 4), tv.TV_ERR_ALIGN), (dict(q_weight=P[3] + 8), tv.TV_ERR_ALIGN),
    (dict(k_weight=P[3] + 8), tv.TV_ERR_ALIGN), (dict(k_out=P[3] + 8), tv.TV_ERR_ALIGN),
    (dict(B=0), tv.TV_OK), (dict(total_rows=0), tv.TV_OK),
])
def test_qk_norm_rope(kw, code):
    assert rc(tv.tv_qk_norm_rope, ROPE, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), tv.TV_ERR_SHAPE), (dict(num_rows=-1), tv.TV_ERR_SHAPE),
    (dict(vocab=0), tv.TV_ERR_SHAPE), (dict(row_stride=99), tv.TV_ERR_SHAPE),
    (dict(rows=None, R=5), tv.TV_ERR_SHAPE), (dict(logits_dtype=2), tv.TV_ERR_DTYPE),
    (dict(scale=0.0), tv.TV_ERR_SHAPE), (dict(scale=-1.0), tv.TV_ERR_SHAPE),
    (dict(scale=float("nan")), tv.TV_ERR_SHAPE), (dict(scale=float("inf")), tv.TV_ERR_SHAPE),
    (dict(top_k=-1), tv.TV_ERR_SHAPE), (dict(top_k=101), tv.TV_ERR_SHAPE),
    (dict(top_k=33), tv.TV_ERR_UNSUPPORTED), (dict(vocab=3, top_k=4), tv.TV_ERR_SHAPE),
    (dict(dev_status=None), tv.TV_ERR_NULL), (dict(tokens=None), tv.TV_ERR_NULL),
    (dict(logprob=None), tv.TV_ERR_NULL), (dict(logits=None), tv.TV_ERR_NULL),
    (dict(top_token=None), tv.TV_ERR_NULL), (dict(top_logprob=None), tv.TV_ERR_NULL),
    (dict(logits=P[0] + 2), tv.TV_ERR_ALIGN), (dict(rows=P[1] + 4), tv.TV_ERR_ALIGN),
    (dict(tokens=P[1] + 4), tv.TV_ERR_ALIGN), (dict(logprob=P[1] + 4), tv.TV_ERR_ALIGN),
    (dict(entropy=P[1] + 4), tv.TV_ERR_ALIGN), (dict(R=0), tv.TV_OK),
    (dict(tokens=None, logprob=None, entropy=None, top_k=0, top_token=None, top_logprob=None),
     tv.TV_OK),
])
def test_logprobs(kw, code):
    assert rc(tv.tv_logprobs, LOGPROBS, **kw) == code


def test_prefill_workspace_of_invalid_sizes():
    f = tv.tv_prefill_workspace_bytes
    assert f(2, 9, 8, 3, 12, 64, 0, 0) == 0 and f(2, 17, 8, 3, 64, 64, 0, 0) == 0
    assert f(0, 0, 8, 3, 64, 64, 0, 0) == 0
    assert f(1, 4000, 4000, 2, 64, 64, 0, 0) % 16 == 0
    assert f(1, 4000, 4000, 2, 64, 64, 0, 1) == 0 and f(1, 4000, 4000, 2, 64, 64, 1, 0) == 0


def test_constants_match_the_header():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "include", "treeverify.h")).read()
    for name in ("TV_ROPE_HALVES", "TV_ROPE_PAIRS", "TV_LOGPROBS_MAX_TOP"):
        m = re.search(r"%s\s*=?\s*(\d+)" % name, src[src.index("enum tv_rope"):])
        assert m and int(m.group(1)) == getattr(tv, name), name
    m = re.search(r"#define TV_PREFILL_TEST_EXPIRE_WAIT\s+(0x[0-9a-f]+)", src)
    assert m and int(m.group(1), 16) == tv.TV_PREFILL_TEST_EXPIRE_WAIT


@pytest.mark.parametrize("f,base,kw", [
    (tv.tv_prefill, PREFILL, dict(total_rows=0x7fff0001, max_rows=0x7fffffff)),
    (tv.tv_qk_norm_rope, ROPE, dict(H=1 << 23, q_stride=1 << 30, q_out_stride=1 << 30)),
])
def test_counts_past_the_limit(f, base, kw):
    assert rc(f, base, **kw) == tv.TV_ERR_UNSUPPORTED
