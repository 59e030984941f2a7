"""tv_prefill on tensor cores at the ends of its range: decays that span a chunk's 120 log2 units,
with sums of products and states far from one.  Bounds are those of recurrence_util.Rows.bounds."""
import numpy as np
import pytest

from recurrence_util import Rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()


@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64), (64, 128), (64, 64)])
@pytest.mark.parametrize("out32", [False, True])
@pytest.mark.parametrize("g,qk,v,state", [(-1.28, 26, 26, 52), (-1.28, 26, -36, -10), (-1.28, -36, 0, -36),
                                          (1.2, 0, 0, 0), (1.2, -36, 0, -36)])
def test_sums_far_from_one(dk, dv, out32, g, qk, v, state):
    """Products of an element of q and one of k of order 2^qk, v of order 2^v, states of order
    2^state; 64 rows span 118 (or 110) log2 units.  The largest sums are 2^52 times the root of dk
    (2^3.5) and a tail of 4 sigma in q . k and v (2^4): below the 2^67 that the header gives for
    such spans.  What is near 2^-36 stays above 2^-42, but for elements next to zero, which the
    magnitude in the bounds covers."""
    import torch
    rng = np.random.default_rng(41)
    r = Rows(rng, [64, 100], 2, dk, dv)
    for name, e, w in (("q", qk // 2, dk), ("k", qk // 2, dk), ("v", v, dv)):
        r.dev[name] = (r.dev[name].float() * (2.0 ** e * np.sqrt(w))).bfloat16()
        r.host[name] = r.dev[name].double().cpu().numpy().reshape(r.host[name].shape)
    r.g.fill_(g)
    if g > 0:  # (growth in one chunk: in two it would leave single precision)
        r.g[64:].zero_()
    r.host["g"] = r.g.cpu().numpy().astype(np.float64)
    x = (rng.normal(size=(r.B, r.H, dk, dv)) * 2.0 ** state).astype(np.float32)
    H0, h0 = torch.from_numpy(x).cuda(), x.astype(np.float64)
    got = r.prefill(H0, out32)
    torch.cuda.synchronize()
    r.check(got, h0, out32)
