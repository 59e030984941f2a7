"""Paths of the serving kernels that only larger calls take: many requests, more items than the
GPU has room for at once, more units than SMs; graphs, streams and threads."""
import numpy as np
import pytest

from recurrence_util import Rows
from test_prefill_gpu import OneRow, WIDTHS, decode
from test_qk_norm_rope_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()


# ---------------------------------------------------------------- norms with rotation


def lengths(seed, B, most):
    n = np.random.default_rng(seed).integers(0, most + 1, B)
    n[[0, B // 2, B - 1]] = 0                      # requests without rows at both ends
    return [int(x) for x in n]


@pytest.mark.parametrize("B", [32, 33, 64, 1024, 1025, 3000])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("trees", [False, True])
def test_rotation_of_many_requests(B, d, trees):
    c = Case(31, lengths(31, B, 3), 2, 1, d, 64, trees=trees, extra=5)
    c.check(c.run())
    assert all(bool(x[c.n:].isnan().all()) for x in c.run())


@pytest.mark.parametrize("B,most", [(7, 2500), (200, 90)])
@pytest.mark.parametrize("d,H,Hkv,f32,pairs", [(128, 40, 20, False, False), (64, 40, 20, False, True),
                                               (256, 16, 5, False, False), (128, 30, 7, True, False),
                                               (64, 33, 1, True, True)])
def test_rotation_of_more_items_than_resident_warps(B, most, d, H, Hkv, f32, pairs):
    import torch
    lens = lengths(32, B, most)
    c = Case(32, lens, H, Hkv, d, d, f32=f32, pairs=pairs, extra=3)
    # items: 256 / d rows and a few heads, four at least, down to where there are twice as many as
    # the 24 (fp32: 16) warps an SM has room for
    resident = torch.cuda.get_device_properties(0).multi_processor_count * (16 if f32 else 24)
    rows, heads = -(-c.R * d // 256), H + Hkv
    per_row = min(max(-(-2 * resident // rows), (heads + 10) // 20), -(-heads // 4))
    per_item = -(-(-(-heads // per_row)) // 4) * 4
    assert rows * -(-heads // per_item) > resident
    outs = c.run()
    c.check(outs)
    assert all(bool(x[c.n:].isnan().all()) for x in outs)


def test_rotation_captured_and_on_another_stream():
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    c = Case(33, lengths(33, 50, 40), 8, 2, 128, 128)
    want = [x.clone() for x in c.run()]
    ints = [torch.from_numpy(x).cuda() for x in (c.offsets, c.start)]
    freq = torch.from_numpy(c.freq).cuda()
    outs, status = [torch.zeros_like(x) for x in want], torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(stream=None):
        tv.tv_qk_norm_rope(c.B, c.R, 8, 2, 128, 128, tv.TV_ROPE_HALVES, tv.TV_BF16, *ints, None,
                           c.dev[0], c.stride[0], c.dev[1], c.stride[1], *c.dw, c.eps, freq, outs[0],
                           c.stride[0], outs[1], c.stride[1], status, stream=stream)

    replayed(call, outs, want)
    assert int(status[0]) == 0


def replayed(call, outs, want):
    """`call` into a graph, replayed twice, and called on a stream, gives `want`."""
    import torch
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    stream = torch.cuda.Stream()
    for go in (graph.replay, graph.replay, lambda: call(stream)):
        for x in outs:
            x.fill_(float("nan"))
        torch.cuda.synchronize()
        go()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


def at_once(calls, want):
    """Two threads, each with a stream, call eight times; every result is what it is alone."""
    import threading

    import torch
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(8):
                got = calls[i](stream)
                stream.synchronize()
                if not all(torch.equal(x, y) for x, y in zip(got, want[i])):
                    bad.append(i)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_rotation_from_two_threads():
    cases = [Case(34, lengths(34, 50, 40), 8, 2, 128, 128), Case(35, [900, 11], 4, 4, 64, 32, f32=True)]
    want = [[x.clone() for x in c.run()] for c in cases]
    at_once([lambda s, c=c: c.run(stream=s) for c in cases], want)


# ---------------------------------------------------------------- single tokens


def decode_call(r, H0, out, H_new, stream=None):
    import tree_speculative_verify_tv_gb300 as tv
    d = r.dev
    tv.tv_decode(r.B, r.H, r.dk, r.dv, tv.TV_DECAY_DIAG if r.diag else tv.TV_DECAY_SCALAR,
                 tv.TV_F32 if r.f32 else tv.TV_BF16, None, H0, d["q"], r.stride["q"], d["k"],
                 r.stride["k"], d["v"], r.stride["v"], r.g, r.g_stride, tv.TV_F32, out, H_new,
                 stream=stream)
    return out, H_new


def test_decode_captured_and_on_another_stream():
    import torch
    r = OneRow(np.random.default_rng(36), [1] * 20, 16, 128, 64)
    H0, _ = r.state(np.random.default_rng(36))
    want = [x.clone() for x in decode(r, H0, True)[:2]]
    outs = [torch.zeros_like(x) for x in want]
    replayed(lambda stream=None: decode_call(r, H0, *outs, stream=stream), outs, want)


def test_decode_from_two_threads():
    import torch
    rows = [OneRow(np.random.default_rng(37 + i), [1] * B, 8, dk, 128, diag=i > 0, f32=i > 0)
            for i, (B, dk) in enumerate([(40, 128), (3, 96)])]
    states = [r.state(np.random.default_rng(38))[0] for r in rows]
    want = [[x.clone() for x in decode(r, H0, True)[:2]] for r, H0 in zip(rows, states)]

    def call(i, s):
        out, H_new = (torch.zeros_like(x) for x in want[i])
        return decode_call(rows[i], states[i], out, H_new, s)

    at_once([lambda s, i=i: call(i, s) for i in range(2)], want)


# ---------------------------------------------------------------- prompts


def chains(r, H0, magnitude):
    """The recurrence in 64 bits on the device, all requests a row at a time (oracle.prefill is the
    same, for less).  With `magnitude`: of absolute values."""
    import torch
    f = (lambda x: x.abs()) if magnitude else (lambda x: x)
    val = {n: f(torch.from_numpy(x).cuda()) for n, x in r.host.items() if n != "g"}
    decay = torch.exp(torch.from_numpy(np.array(r.host["g"])).cuda())
    out = torch.zeros(r.R, r.H, r.dv, dtype=torch.float64, device="cuda")
    S = f(H0.double()).clone()
    order = np.argsort(-np.array(r.lens), kind="stable")
    lens = np.array(r.lens)[order]
    first = torch.from_numpy(r.offsets[:-1][order].astype(np.int64)).cuda()
    S = S[torch.from_numpy(order).cuda()]
    for t in range(int(lens[0])):
        n = int((lens > t).sum())
        at = first[:n] + t
        S[:n] = decay[at][..., None, None] * S[:n] + val["k"][at][..., None] * val["v"][at][:, :, None]
        out[at] = torch.einsum("bhc,bhcd->bhd", val["q"][at], S[:n])
    back = torch.empty_like(S)
    back[torch.from_numpy(order).cuda()] = S
    return out, back


def check_prompts(r, H0, got, out32):
    import torch
    rel, absolute, sabs = r.bounds(out32)
    (want, state), (mag, smag) = chains(r, H0, False), chains(r, H0, True)
    out, H_new, status = got
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    tiny = 1e-30
    assert ((out.double() - want).abs() <= rel * want.abs() + absolute * mag + tiny).all()
    assert ((H_new.double() - state).abs() <= sabs * smag + tiny).all()


@pytest.mark.parametrize("dk,dv", WIDTHS)
@pytest.mark.parametrize("out32", [False, True])
@pytest.mark.parametrize("B", [45, 70])
def test_more_units_than_sms(dk, dv, out32, B):
    """Units that CTAs take over from others that have not been launched, with requests in order of
    length (up to 64) or as they come."""
    import torch
    rng = np.random.default_rng(39)
    lens = [int(x) for x in rng.integers(0, 260, B)]
    lens[3], lens[B - 1], lens[B // 2] = 0, 700, 650
    H = -(-3 * torch.cuda.get_device_properties(0).multi_processor_count // B)
    r = Rows(rng, lens, H, dk, dv)
    H0, _ = r.state(rng)
    check_prompts(r, H0, r.prefill(H0, out32), out32)


@pytest.mark.parametrize("dk,dv", WIDTHS)
@pytest.mark.parametrize("out32", [False, True])
def test_more_segments_than_sms(dk, dv, out32):
    """Prompts in so many segments that the launch of their sums takes items over too."""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    H, lens = 19, [5000, 4700, 4990]
    rng = np.random.default_rng(40)
    r = Rows(rng, lens, H, dk, dv, decay=0.05)
    H0, _ = r.state(rng)
    size = tv.tv_prefill_workspace_bytes(3, r.R, 5000, H, dk, dv, tv.TV_DECAY_SCALAR, tv.TV_BF16)
    pieces = size // (3 * H * (dk * dv * 4 + 8))
    assert (pieces - 1) * 3 * H > sms
    check_prompts(r, H0, r.prefill(H0, out32, workspace=True), out32)
