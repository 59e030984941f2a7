"""tv_prefill and tv_decode against the recurrence in 64 bits, row after row.  The bounds are
those that recurrence_util.Rows.bounds derives from the arithmetic."""
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


def run(seed, lens, H, dk, dv, out32=True, state=False, **kw):
    import torch
    rng = np.random.default_rng(seed)
    call = {n: kw.pop(n) for n in ("max_rows", "workspace") if n in kw}
    r = Rows(rng, lens, H, dk, dv, **kw)
    H0, h0 = r.state(rng) if state else (None, None)
    got = r.prefill(H0, out32, **call)
    torch.cuda.synchronize()
    r.check(got, h0, out32)
    return r, got


WIDTHS = [(128, 128), (128, 64), (64, 128), (64, 64)]


@pytest.mark.parametrize("dk,dv", WIDTHS)
@pytest.mark.parametrize("out32", [False, True])
@pytest.mark.parametrize("lens", [[1], [64], [65, 0, 63], [130, 1, 200, 64, 128, 2]])
def test_lengths_around_a_chunk(dk, dv, out32, lens):
    run(1, lens, 3, dk, dv, out32, state=True)


@pytest.mark.parametrize("dk,dv", [(16, 16), (8, 256), (40, 24), (256, 8), (128, 128), (96, 64)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("diag", [False, True])
def test_widths_types_and_decays(dk, dv, f32, diag):
    run(2, [17, 0, 8, 9, 70], 2, dk, dv, out32=f32, state=True, f32=f32, diag=diag)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("gates", ["token", "head"])
@pytest.mark.parametrize("kind", ["tensor", "f32", "diag"])
def test_strides_and_shared_decays(fused, gates, kind):
    run(3, [100, 31, 70], 4, 128, 64, state=False, fused=fused, gates=gates, f32=kind == "f32",
        diag=kind == "diag")


@pytest.mark.parametrize("decay", [0.0, 1e-4, 0.02, 5.0, 60.0])
@pytest.mark.parametrize("dk,dv", [(128, 64), (64, 128)])
def test_slow_and_fast_decays(decay, dk, dv):
    run(4, [700, 129], 2, dk, dv, state=True, decay=decay)


def test_growing_states():
    """g > 0 is allowed: states that grow."""
    run(5, [200, 40], 2, 128, 128, state=True, decay=-0.05)


@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("lens,H", [([3000], 1), ([1500, 20, 2900, 64], 2), ([4097], 3)])
@pytest.mark.parametrize("workspace", [True, 0])
def test_long_prompts_with_and_without_cuts(dk, dv, lens, H, workspace):
    run(6, lens, H, dk, dv, state=True, workspace=workspace, decay=0.1)


def test_a_small_workspace_cuts_less():
    import tree_speculative_verify_tv_gb300 as tv
    need = tv.tv_prefill_workspace_bytes(1, 4000, 4000, 2, 64, 128, tv.TV_DECAY_SCALAR, tv.TV_BF16)
    for part in (need // 2, need // 5, 16):
        run(7, [4000], 2, 64, 128, state=True, workspace=max(16, part // 16 * 16), decay=0.1)


def test_single_precision_outputs_keep_it():
    """Normwise: the error of the outputs and of the state stays near single precision, with
    decays that let 2000 rows add up."""
    import torch
    rng = np.random.default_rng(8)
    r = Rows(rng, [2500, 600], 2, 128, 128, gates="head", decay=5e-4)
    out, H_new, _ = r.prefill()
    want, state = r.reference()
    torch.cuda.synchronize()
    for x, y in ((out, want), (H_new, state)):
        x = x.cpu().numpy().astype(np.float64)
        assert np.linalg.norm(x - y) <= 1e-6 * np.linalg.norm(y)


def test_cuts_without_a_state():
    run(24, [4000, 130], 2, 64, 64, out32=False, decay=0.02)


def test_two_streams_and_threads():
    """Calls at the same time, each with a workspace of its own, give what they give alone."""
    import threading

    import torch
    rows = [Rows(np.random.default_rng(25 + i), lens, 2, 128, dv) for i, (lens, dv) in
            enumerate([([2000, 5], 64), ([64] * 9, 128)])]
    want = [[x.clone() for x in r.prefill()[:2]] for r in rows]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(8):
                got = rows[i].prefill(stream=stream)
                stream.synchronize()
                if int(got[2][0]) or not all(torch.equal(x, y) for x, y in zip(want[i], got)):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_resets_and_mixed_decays():
    """Rows that forget everything (as between packed documents: -inf, or so large that 2^4096 is
    left behind), beside rows that keep all of it."""
    import torch
    rng = np.random.default_rng(27)
    r = Rows(rng, [300, 64], 2, 128, 64)
    g = r.g.clone()
    g[:] = 0.0
    g[50], g[51], g[130], g[191], g[320, 1] = -3000.0, -200.0, -1e30, -float("inf"), -float("inf")
    g[200:240] = -2.5
    r.g, r.host["g"] = g, g.cpu().numpy().astype(np.float64)
    H0, h0 = r.state(rng)
    for out32 in (False, True):
        got = r.prefill(H0, out32)
        torch.cuda.synchronize()
        r.check(got, h0, out32)


def test_max_rows_is_only_a_bound():
    for max_rows in (200, 1000, 1 << 20):
        run(9, [200, 150], 2, 128, 128, max_rows=max_rows)


@pytest.mark.parametrize("dk", [64, 40])
def test_in_place_and_in_pieces(dk):
    """A prompt in three calls, the state in place, gives what one call gives."""
    import torch
    rng = np.random.default_rng(10)
    r = Rows(rng, [333], 2, dk, 64)
    H0, h0 = r.state(rng)
    H = H0.clone()
    outs, at = [], 0
    for n in (100, 1, 232):
        p = Rows(np.random.default_rng(0), [n], 2, dk, 64)
        p.dev = {x: y[at:at + n] for x, y in r.dev.items()}
        p.g = r.g[at:at + n]
        p.stride, p.g_stride = r.stride, r.g_stride
        outs.append(p.prefill(H, H_new=H)[0])
        at += n
    torch.cuda.synchronize()
    r.check((torch.cat(outs), H, torch.zeros(1)), h0)


def test_decays_past_any_count_over_many_rows():
    """Half a million rows a segment that each leave 2^4096 behind: the segment's decay is 0, although
    its logarithm is past what a 64-bit sum of 2^-32 holds.  An output is its own row's product."""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    n, d = (1 << 20) + 128, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(n, d, generator=gen, device="cuda").bfloat16() for _ in range(3))
    H0 = torch.randn(1, 1, d, d, generator=gen, device="cuda")
    g = torch.full((1,), -float("inf"), device="cuda")
    out = torch.full((n, 1, d), float("nan"), device="cuda")
    H_new, status = torch.full_like(H0, float("nan")), torch.zeros(1, dtype=torch.int32, device="cuda")
    size = 2 * (d * d * 4 + 8)  # for two segments
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    tv.tv_prefill(1, n, n, 1, d, d, tv.TV_DECAY_SCALAR, tv.TV_BF16,
                  torch.tensor([0, n], dtype=torch.int32, device="cuda"), H0, q, d, k, d, v, d, g, 0,
                  tv.TV_F32, out, H_new, ws, size, status)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    q, k, v = q.double(), k.double(), v.double()
    want = (q * k).sum(1, keepdim=True) * v
    # 64 products accumulated (2^-23 a step of 16 and its inside), three parts of the weight
    bound = 2.0 ** -19 * (q * k).abs().sum(1, keepdim=True) * v.abs()
    assert ((out[:, 0] - want).abs() <= bound).all()
    state = k[-1][:, None] * v[-1][None]
    assert ((H_new[0, 0] - state).abs() <= 2.0 ** -22 * state.abs()).all()


def test_in_place_with_cuts():
    import torch
    rng = np.random.default_rng(11)
    r = Rows(rng, [5000, 90], 1, 128, 128, decay=0.05)
    H0, h0 = r.state(rng)
    got = r.prefill(H0, H_new=H0)
    torch.cuda.synchronize()
    r.check(got, h0)


@pytest.mark.parametrize("kind", ["tensor", "f32"])
def test_rows_behind_the_last_request_stay(kind):
    import torch
    rng = np.random.default_rng(12)
    r = Rows(rng, [70, 5], 2, 64, 64, f32=kind == "f32", extra=9)
    got = r.prefill()
    torch.cuda.synchronize()
    r.check(got)
    assert torch.isnan(got[0][75:]).all()


@pytest.mark.parametrize("kind", ["tensor", "f32", "diag"])
@pytest.mark.parametrize("what", ["q", "k", "v", "g", "H0"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_value_stays_in_its_request_and_head(kind, what, value):
    """A NaN or an infinity in the first row of the middle request (or its state), head 1: the
    neighbours and the other heads are what they are without it."""
    import torch
    rng = np.random.default_rng(13)
    r = Rows(rng, [40, 70, 33], 3, 64, 64, f32=kind == "f32", diag=kind == "diag")
    H0, _ = r.state(rng)
    clean = [x.clone() for x in r.prefill(H0)[:2]]
    if what == "H0":
        H0[1, 1, 5, 7] = value
    elif what == "g":
        r.g[40].view(3, -1)[1, 0] = value
    else:
        r.dev[what][40].view(3, -1)[1, 3] = value
    out, H_new, status = r.prefill(H0)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    touched = torch.zeros_like(out, dtype=torch.bool)
    touched[40:110, 1] = True
    assert torch.equal(out[~touched], clean[0][~touched])
    assert not torch.isfinite(out[40, 1]).all()
    keep = torch.ones(3, 3, dtype=torch.bool)
    keep[1, 1] = False
    assert torch.equal(H_new[keep], clean[1][keep])


@pytest.mark.parametrize("dk,dv", WIDTHS + [(40, 24)])
@pytest.mark.parametrize("out32", [False, True])
@pytest.mark.parametrize("lens,workspace", [([20, 150, 9], True), ([3000], True)])
def test_a_bad_value_of_v_stays_in_its_column(dk, dv, out32, lens, workspace):
    """NaN and infinities in three columns of v: those columns are no numbers from their rows on (in
    the state too; on tensor cores up to 63 rows ahead of them may be none either), all else is
    what it is without them."""
    import torch
    rng = np.random.default_rng(30)
    r = Rows(rng, lens, 2, dk, dv)
    H0, _ = r.state(rng)
    clean = [x.clone() for x in r.prefill(H0, out32, workspace=workspace)[:2]]
    b = len(lens) // 2
    first, end = int(r.offsets[b]), int(r.offsets[b + 1])
    bad, near = (torch.zeros_like(clean[0], dtype=torch.bool) for _ in range(2))
    v = r.dev["v"].view(r.R, 2, dv)
    for row, col, value in ((37, 5, float("nan")), (70, 20, float("inf")), (63, dv - 1, -float("inf")),
                            (130, 5, float("inf"))):
        v[first + row, 1, col] = value
        bad[first + row:end, 1, col] = True
        if r.tensor_cores():
            near[first + max(0, row - 63):first + row, 1, col] = True
    out, H_new, status = r.prefill(H0, out32, workspace=workspace)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    assert not torch.isfinite(out[bad]).any()
    assert torch.equal(out[~bad & ~near], clean[0][~bad & ~near])
    lost = torch.zeros_like(H_new, dtype=torch.bool)
    lost[b, 1][:, [5, 20, dv - 1]] = True
    assert not torch.isfinite(H_new[lost]).any() and torch.equal(H_new[~lost], clean[1][~lost])


@pytest.mark.parametrize("kind", ["tensor", "f32"])
@pytest.mark.parametrize("offsets", [[0, 50, 20, 90], [-1, 30, 60, 90], [0, 30, 60, 500]])
def test_unusable_offsets(kind, offsets):
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    rng = np.random.default_rng(14)
    r = Rows(rng, [30, 30, 30], 2, 64, 64, f32=kind == "f32")
    r.offsets = np.array(offsets, np.int32)
    _, H_new, status = r.prefill(max_rows=80)
    torch.cuda.synchronize()
    assert int(status[0]) == tv.TV_ERR_TREE
    for b in range(3):
        n = offsets[b + 1] - offsets[b]
        if offsets[b] < 0 or n < 0 or n > 80 or offsets[b + 1] > 90:
            assert torch.isnan(H_new[b]).all()


def test_more_rows_than_the_bound():
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    rng = np.random.default_rng(15)
    r = Rows(rng, [100, 20], 2, 64, 64)
    out, H_new, status = r.prefill(max_rows=99)
    torch.cuda.synchronize()
    assert int(status[0]) == tv.TV_ERR_TREE
    assert torch.isnan(out[:100]).all() and torch.isnan(H_new[0]).all()
    assert torch.isfinite(out[100:]).all() and torch.isfinite(H_new[1]).all()


def test_no_rows_at_all():
    """Requests without rows keep their states, or get zeros."""
    import torch
    rng = np.random.default_rng(16)
    for dk in (64, 24):
        r = Rows(rng, [0, 0], 2, dk, 64)
        H0, _ = r.state(rng)
        _, H_new, status = r.prefill(H0, max_rows=1)
        _, fresh, _ = r.prefill(None, max_rows=1)
        torch.cuda.synchronize()
        assert int(status[0]) == 0 and torch.equal(H_new, H0) and not fresh.any()


def test_many_requests():
    run(17, [int(x) for x in np.random.default_rng(17).integers(0, 40, 300)], 1, 64, 64,
        state=True)


@pytest.mark.parametrize("B,H", [(33, 5), (64, 3), (32, 6), (65, 3)])
def test_requests_of_all_lengths(B, H):
    """More units than SMs: the longest requests go first (up to 64 requests), among them equal and
    empty ones."""
    lens = [int(x) for x in np.random.default_rng(B).integers(0, 200, B)]
    lens[B // 2], lens[3], lens[7], lens[B - 1] = 700, 0, lens[5], 520
    run(28, lens, H, 64, 64, state=True)


def test_an_unusable_request_among_many():
    """One request with more rows than the bound, where the order of the others goes by lengths."""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    rng = np.random.default_rng(29)
    lens = [int(x) for x in rng.integers(1, 90, 40)]
    lens[11], lens[30] = 600, 530
    r = Rows(rng, lens, 4, 64, 64)
    want = r.prefill()
    out, H_new, status = r.prefill(max_rows=560)
    torch.cuda.synchronize()
    assert int(status[0]) == tv.TV_ERR_TREE
    rows = torch.zeros(r.R, dtype=torch.bool)
    rows[int(r.offsets[11]):int(r.offsets[12])] = True
    assert torch.isnan(out[rows]).all() and torch.isnan(H_new[11]).all()
    assert torch.equal(out[~rows], want[0][~rows])
    keep = torch.arange(40) != 11
    assert torch.equal(H_new[keep], want[1][keep])


def test_the_same_call_gives_the_same_bits():
    import torch
    rng = np.random.default_rng(18)
    r = Rows(rng, [3000, 77], 2, 128, 64)
    first = [x.clone() for x in r.prefill()[:2]]
    for _ in range(3):
        again = r.prefill()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_captured_and_on_another_stream():
    import torch
    rng = np.random.default_rng(19)
    r = Rows(rng, [1500, 77], 2, 128, 64)
    want = [x.clone() for x in r.prefill()[:2]]
    torch.cuda.synchronize()
    import tree_speculative_verify_tv_gb300 as tv
    need = tv.tv_prefill_workspace_bytes(2, r.R, 1500, 2, 128, 64, 0, 0)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    out, H_new = (torch.zeros_like(x) for x in want)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    offsets = torch.from_numpy(r.offsets).cuda()

    def call():
        tv.tv_prefill(2, r.R, 1500, 2, 128, 64, 0, 0, offsets, None, r.dev["q"], r.stride["q"],
                      r.dev["k"], r.stride["k"], r.dev["v"], r.stride["v"], r.g, r.g_stride,
                      tv.TV_F32, out, H_new, ws, need, status)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    for _ in range(2):
        out.zero_(), H_new.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(H_new, want[1])
    out.zero_(), H_new.zero_()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    stream.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(H_new, want[1]) and int(status[0]) == 0


# ---------------------------------------------------------------- single tokens


def decode(r, H0, out32, active=None, H_new=None):
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    out = torch.full((r.B, r.H, r.dv), float("nan"), device="cuda",
                     dtype=torch.float32 if out32 else torch.bfloat16)
    if H_new is None:
        H_new = torch.full_like(H0, float("nan"))
    d = r.dev
    tv.tv_decode(r.B, r.H, r.dk, r.dv, tv.TV_DECAY_DIAG if r.diag else tv.TV_DECAY_SCALAR,
                 tv.TV_F32 if r.f32 else tv.TV_BF16, active, H0, d["q"], r.stride["q"], d["k"],
                 r.stride["k"], d["v"], r.stride["v"], r.g, r.g_stride,
                 tv.TV_F32 if out32 else tv.TV_BF16, out, H_new)
    return out, H_new, torch.zeros(1)


class OneRow(Rows):
    def tensor_cores(self):
        return False


@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64), (64, 64), (8, 8), (256, 256), (40, 24),
                                   (16, 200)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("diag", [False, True])
@pytest.mark.parametrize("B,H", [(1, 1), (5, 3), (40, 9)])
def test_decode(dk, dv, f32, diag, B, H):
    rng = np.random.default_rng(20)
    r = OneRow(rng, [1] * B, H, dk, dv, f32=f32, diag=diag, fused=B == 5,
               gates="head" if H == 3 else "token")
    H0, h0 = r.state(rng)
    r.check(decode(r, H0, f32), h0, f32)
    r.check(decode(r, H0, True, H_new=H0), h0, True)  # in place


def test_decode_leaves_inactive_requests():
    import torch
    rng = np.random.default_rng(21)
    r = OneRow(rng, [1] * 6, 4, 128, 64)
    H0, _ = r.state(rng)
    full = decode(r, H0, True)
    active = torch.tensor([1, 0, 1, 0, 0, 7], dtype=torch.int32, device="cuda")
    out, H_new, _ = decode(r, H0, True, active)
    torch.cuda.synchronize()
    on = active.bool()
    assert torch.equal(out[on], full[0][on]) and torch.equal(H_new[on], full[1][on])
    assert torch.isnan(out[~on]).all() and torch.isnan(H_new[~on]).all()


def test_decode_goes_on_from_a_prompt():
    """A prompt of 70 rows gives what 64 rows and six decoding steps give."""
    import torch
    rng = np.random.default_rng(22)
    r = Rows(rng, [70], 3, 128, 64)
    want, state = r.reference()
    p = Rows(np.random.default_rng(0), [64], 3, 128, 64)
    p.dev, p.g, p.stride = {x: y[:64] for x, y in r.dev.items()}, r.g[:64], r.stride
    out, H, _ = p.prefill()
    outs = [out]
    for t in range(64, 70):
        s = OneRow(np.random.default_rng(0), [1], 3, 128, 64)
        s.dev, s.g, s.stride = {x: y[t:t + 1] for x, y in r.dev.items()}, r.g[t].clone(), r.stride
        outs.append(decode(s, H, True, H_new=H)[0])
    torch.cuda.synchronize()
    r.check((torch.cat(outs), H, torch.zeros(1)))


# ---------------------------------------------------------------- the timeout path


def test_expired_waits_are_reported_and_leave_the_gpu_usable():
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    rng = np.random.default_rng(23)
    r = Rows(rng, [300, 77], 2, 128, 64)
    want = [x.clone() for x in r.prefill()[:2]]
    out, H_new = (torch.zeros_like(x) for x in want)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tv.tv_prefill(2, r.R, 300, 2, 128, 64, 0, 0, torch.from_numpy(r.offsets).cuda(), None,
                  r.dev["q"], r.stride["q"], r.dev["k"], r.stride["k"], r.dev["v"], r.stride["v"],
                  r.g, r.g_stride, tv.TV_F32 | tv.TV_PREFILL_TEST_EXPIRE_WAIT, out, H_new, None, 0,
                  status)
    torch.cuda.synchronize()
    assert int(status[0]) == tv.TV_ERR_TIMEOUT
    again = r.prefill()
    torch.cuda.synchronize()
    assert int(again[2][0]) == 0 and all(torch.equal(x, y) for x, y in zip(want, again))
