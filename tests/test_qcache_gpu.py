"""GPU parity of the 4-bit KV cache.

The cache itself is compared byte for byte with the oracle's quantiser: steps and codes
are defined by exact quotients, so there is nothing to tolerate.  Read-back values are
exact in bf16 and compared for equality.

Attention's bound, per output row, from the arithmetic (u = 2^-23 bounds one fp32
operation, truncating accumulation included): a score scale * sum_c q_c k_c of magnitude
at most smax = scale * max_j sum_c |q_c k_c| goes through d / 16 accumulation steps, two
further roundings and the base-2 exponential (2 u, and its argument's rounding, the
magnitude of the score and of the reference maximum each): weights carry a relative error
of e = (d / 16 + 6) * 2 u smax + 8 u, plus 2^-16 for their bf16 hi + lo split.  Numerator
and denominator are sums of n weighted values in any order of blocks of 16 (n / 16 + 16
steps of u); with all |v| <= vmax a row is off by at most
    vmax * 2 * (e + 2^-16 + (n / 16 + 16) u),
plus the output's own rounding: |o| * 2^-8 in bf16, |o| * 2^-24 in fp32.
"""
import numpy as np
import pytest

import oracle
import workloads

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()


def cu(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.view(dtype)).cuda()


def bf(x):
    """float array -> (device bf16 tensor, its exact float32 values)."""
    import torch
    bits = workloads.f32_to_bf16_bits(np.asarray(x, np.float32))
    return cu(bits, torch.bfloat16), workloads.bf16_bits_to_f32(bits)


def status(st):
    import torch
    torch.cuda.synchronize()
    return int(st[0])


class Cache:
    """A cache on the device, its copy on the host and its page table."""

    def __init__(self, rng, B, max_pages, Hkv, d, fill=None):
        import tree_speculative_verify_tv_gb300 as tv
        self.B, self.mp, self.Hkv, self.d = B, max_pages, Hkv, d
        self.table, self.pages = workloads.qcache_pages(rng, B, max_pages)
        rec = tv.tv_qcache_bytes(1, 1, d)
        shape = (self.pages, Hkv, rec)
        self.host = np.full(shape, fill, np.uint8) if fill is not None else \
            rng.integers(0, 256, shape).astype(np.uint8)
        self.dev = cu(self.host)
        self.dev_table = cu(self.table)

    def put(self, b, pos, k, v):
        """Row k, v [Hkv][d] into the host copy."""
        for h in range(self.Hkv):
            oracle.qcache_put(self.host[self.table[b, pos // 64], h], self.d, pos % 64, k[h], v[h])

    def values(self):
        """K, V as [B][Hkv][positions][d] from the host copy."""
        K, V = oracle.qcache_get(self.host[self.table], self.d)  # [B, mp, Hkv, 64, d]
        f = lambda x: x.transpose(0, 2, 1, 3, 4).reshape(self.B, self.Hkv, -1, self.d)  # noqa: E731
        return f(K), f(V)

    def fetch(self):
        return self.dev.cpu().numpy()


def strided(rng, rows, widths, pad):
    """bf16 views of row-major blocks side by side in one tensor: [(view, values)], stride."""
    total = sum(widths) + pad
    base, val = bf(rng.normal(size=(max(rows, 1), total)))
    out, at = [], 0
    for w in widths:
        out.append((base[:, at:at + w], val[:rows, at:at + w]))
        at += w
    return out, total


def write(c, rng, lens, start, pad=0, k=None, v=None, stream=None):
    """tv_qcache_write of random (or given) rows; the host copy follows."""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    lens, start = np.asarray(lens, np.int32), np.asarray(start, np.int32)
    R, w = int(lens.sum()), c.Hkv * c.d
    offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    if k is None:
        ((dk, k), (dv, v)), stride = strided(rng, R, [w, w], pad)
    else:
        (dk, k), (dv, v), stride = bf(k), bf(v), w
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tv.tv_qcache_write(c.B, R, c.Hkv, c.d, c.pages, c.mp, cu(offs), cu(start), c.dev_table, dk,
                       dv, stride, c.dev, st, stream=stream)
    assert status(st) == 0
    for b in range(c.B):
        for m in range(lens[b]):
            r = offs[b] + m
            c.put(b, int(start[b]) + m, k[r].reshape(c.Hkv, c.d), v[r].reshape(c.Hkv, c.d))


def read(c, lens, start, ctx, pad=0, check=0, table=None, offs=None):
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    lens = np.asarray(lens, np.int32)
    R, w = int(lens.sum()), c.Hkv * c.d
    if offs is None:
        offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    base = torch.full((max(R, 1), 2 * w + pad), 77.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tv.tv_qcache_read(c.B, R, c.Hkv, c.d, c.pages, c.mp, cu(offs), cu(np.asarray(start, np.int32)),
                      cu(np.asarray(ctx, np.int32)), c.dev_table if table is None else cu(table),
                      c.dev, base[:, :w], base[:, w:], 2 * w + pad, st)
    assert status(st) == check
    assert bool((base[:, 2 * w:] == 77).all())
    f = lambda x: x[:R].float().cpu().numpy().reshape(R, c.Hkv, c.d)  # noqa: E731
    return f(base[:, :w]), f(base[:, w:2 * w])


# ---------------------------------------------------------------- write and read


@pytest.mark.parametrize("d,Hkv,lens,start,pad", [
    (128, 2, [1], [0], 0), (128, 1, [64], [0], 8), (64, 3, [5, 0, 64, 130], [59, 3, 32, 0], 24),
    (128, 8, [7, 1, 9], [1, 63, 64], 0), (64, 1, [200, 1], [13, 191], 0), (64, 2, [2, 3], [6, 7], 8),
    (128, 2, [0, 65, 0], [0, 127, 5], 0),
])
def test_write_is_the_definition_byte_for_byte(d, Hkv, lens, start, pad):
    rng = np.random.default_rng(d + sum(lens))
    c = Cache(rng, len(lens), 4, Hkv, d)
    write(c, rng, lens, start, pad)
    assert np.array_equal(c.fetch(), c.host)


def test_rows_written_one_at_a_time_equal_rows_written_at_once():
    rng = np.random.default_rng(2)
    one, all_ = Cache(rng, 1, 3, 2, 64, fill=0), None
    rows = rng.normal(size=(2, 75, 128))
    for m in range(75):
        write(one, rng, [1], [40 + m], k=rows[0][m:m + 1], v=rows[1][m:m + 1])
    all_ = Cache(np.random.default_rng(2), 1, 3, 2, 64, fill=0)
    write(all_, rng, [75], [40], k=rows[0], v=rows[1])
    assert np.array_equal(one.fetch(), all_.fetch())


def test_ties_zeros_tiny_huge_and_not_finite():
    rng = np.random.default_rng(3)
    c = Cache(rng, 1, 2, 1, 64)
    k, v = rng.normal(size=(2, 70, 64))
    for x in (k, v):
        for r in range(32):  # every step's halves: ties of the code, and ties of the step
            s = (8 + r % 8) * 2.0 ** (r // 8 - 4)
            x[r, :32] = s * (np.arange(32) % 15 - 7) / 2
            x[r, 0] = 7 * s
            x[r, 32:] = np.linspace(-1, 1, 32) * 7 * (2 * (r % 8) + 17) * 2.0 ** -4
        x[32] = 0
        x[33] *= 1e-12
        x[34] *= 1e-38
        x[35] *= 1e4
        x[36, 5], x[37, 40], x[38, 0] = np.inf, -np.inf, 3e38
        x[39, 2] = -6272.0
        x[40, :32] = -0.0
    write(c, rng, [70], [3], k=k, v=v)
    assert np.array_equal(c.fetch(), c.host)
    k[41, 7], v[42, 33] = np.nan, np.nan  # the scale says so; the group's codes are free
    write(c, rng, [70], [3], k=k, v=v)
    gk, gv = read(c, [70], [3], [73])
    wk, wv = (x[0, :, 3:73].transpose(1, 0, 2) for x in c.values())
    np.testing.assert_array_equal(gk, wk)
    np.testing.assert_array_equal(gv, wv)
    assert np.isnan(gk[41, 0, :32]).all() and np.isfinite(gk[41, 0, 32:]).all()
    assert np.isnan(gv[42, 0, 32:]).all() and np.isfinite(gv[42, 0, :32]).all()


@pytest.mark.parametrize("d,Hkv,lens,start,ctx,pad", [
    (128, 2, [64, 1, 100], [0, 63, 17], [64, 64, 60], 0), (64, 3, [5, 0, 90], [60, 0, 100], [64, 9, 192], 8),
    (128, 1, [192], [0], [0], 0), (64, 1, [3], [189], [192], 40),
])
def test_read_gives_the_values_and_zeros_past_the_context(d, Hkv, lens, start, ctx, pad):
    rng = np.random.default_rng(sum(lens))
    c = Cache(rng, len(lens), 3, Hkv, d)
    gk, gv = read(c, lens, start, ctx, pad)
    K, V = c.values()
    at = 0
    for b, n in enumerate(lens):
        for m in range(n):
            pos = start[b] + m
            live = pos < ctx[b]
            for got, held in ((gk, K), (gv, V)):
                np.testing.assert_array_equal(got[at], held[b, :, pos] if live else np.zeros((Hkv, d)))
            at += 1


def test_bad_rows_write_nothing_and_read_zeros():
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    rng = np.random.default_rng(5)
    c = Cache(rng, 3, 2, 2, 64)
    k, _ = bf(rng.normal(size=(30, 128)))
    offs = np.array([0, 10, 20, 30], np.int32)

    def wr(offs, start, table):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        tv.tv_qcache_write(3, 30, 2, 64, c.pages, 2, cu(np.asarray(offs, np.int32)),
                           cu(np.asarray(start, np.int32)), cu(table), k, k, 128, c.dev, st)
        return status(st)

    before = c.fetch()
    far = c.table.copy()
    far[:, :] = -1
    assert wr(offs, [0, 0, 0], far) == tv.TV_ERR_SHAPE
    far[:, :] = c.pages
    assert wr(offs, [0, 0, 0], far) == tv.TV_ERR_SHAPE
    assert wr(offs, [119, -1, 2 ** 31 - 1], c.table) == tv.TV_ERR_SHAPE
    assert wr([0, 31, 31, 31], [0, 0, 0], c.table) == tv.TV_ERR_TREE
    assert wr([-5, -1, -9, -20], [0, 0, 0], c.table) == tv.TV_ERR_TREE
    assert np.array_equal(c.fetch(), before)
    # one bad request of three: the others are served
    gk, _ = read(c, [10, 10, 10], [0, 120, 5], [128, 128, 128], check=tv.TV_ERR_SHAPE)
    K, _ = c.values()
    np.testing.assert_array_equal(gk[:10], K[0, :, :10].transpose(1, 0, 2))
    assert np.all(gk[10:20] == 0)
    np.testing.assert_array_equal(gk[20:], K[2, :, 5:15].transpose(1, 0, 2))
    gk, gv = read(c, [10, 10, 10], [0, 0, 5], [128, 129, -1], check=tv.TV_ERR_SHAPE)
    assert np.all(gk[10:] == 0) and np.all(gv[10:] == 0) and np.abs(gk[:10]).max() > 0
    bad = c.table.copy()
    bad[1, 0] = c.pages + 7
    gk, _ = read(c, [10, 10, 10], [0, 60, 5], [128, 128, 128], check=tv.TV_ERR_SHAPE, table=bad)
    assert np.all(gk[10:14] == 0)
    np.testing.assert_array_equal(gk[14:20], K[1, :, 64:70].transpose(1, 0, 2))


def test_pages_past_four_gigabytes():
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    rng = np.random.default_rng(6)
    Hkv, d, pages = 8, 128, 66000  # 4.6 GB
    assert tv.tv_qcache_bytes(pages, Hkv, d) > 1 << 32
    dev = torch.empty(tv.tv_qcache_bytes(pages, Hkv, d), dtype=torch.uint8, device="cuda")
    small = Cache(rng, 1, 2, Hkv, d, fill=0)
    small.table = np.array([[0, 1]], np.int32)
    tall = np.array([[pages - 1, pages - 2]], np.int32)
    k, kv = bf(rng.normal(size=(70, Hkv * d)))
    offs, st = cu(np.array([0, 70], np.int32)), torch.zeros(1, dtype=torch.int32, device="cuda")
    z, n = cu(np.array([10], np.int32)), cu(np.array([80], np.int32))
    tv.tv_qcache_write(1, 70, Hkv, d, pages, 2, offs, z, cu(tall), k, k, Hkv * d, dev, st)
    out = torch.zeros((2, 70, Hkv * d), dtype=torch.bfloat16, device="cuda")
    tv.tv_qcache_read(1, 70, Hkv, d, pages, 2, offs, z, n, cu(tall), dev, out[0], out[1], Hkv * d, st)
    assert status(st) == 0
    want = oracle.qcache_values(*oracle.qcache_quantise(kv))
    for i in (0, 1):
        np.testing.assert_array_equal(out[i].float().cpu().numpy(), want)
    # attention over those pages
    q, qv = bf(rng.normal(size=(1, 16, d)))
    kt, ktv = bf(rng.normal(size=(1, Hkv, d)))
    o = torch.zeros((1, 16, d), dtype=torch.float32, device="cuda")
    wsb = tv.tv_qcache_attention_workspace_bytes(1, 1, 1, 16, Hkv, d, 2)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device="cuda")
    ctx = cu(np.array([80], np.int32))
    par = cu(np.array([-1], np.int32))
    tv.tv_qcache_write(1, 10, Hkv, d, pages, 2, cu(np.array([0, 10], np.int32)),
                       cu(np.array([0], np.int32)), cu(tall), k, k, Hkv * d, dev, st)
    tv.tv_qcache_attention(1, 1, 1, 16, Hkv, d, pages, 2, cu(np.array([0, 1], np.int32)), par, ctx,
                           cu(tall), 0, 0, q, 16 * d, dev, kt, kt, Hkv * d, 0.1, tv.TV_F32, o, ws,
                           wsb, st)
    assert status(st) == 0
    held = np.concatenate([want[:10], want]).reshape(1, 80, Hkv, d).transpose(0, 2, 1, 3)
    check_rows(o.cpu().numpy(), np.array([0, 1]), np.array([-1]), qv, held, held, [80], ktv, ktv,
               0.1, 0, 0, False)


# ---------------------------------------------------------------- commit


def commit(c, b, ctx, lens, path, kt, vt, stride, in_place=False, table=None, expect=0):
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dctx = cu(np.asarray(ctx, np.int32))
    new = dctx if in_place else torch.full_like(dctx, -7)
    tv.tv_qcache_commit(b.B, b.T, b.max_nodes, path.shape[1], c.Hkv, c.d, c.pages, c.mp,
                        cu(b.node_offsets), cu(path), cu(lens), dctx,
                        c.dev_table if table is None else cu(table), kt, vt, stride, c.dev, new, st)
    assert status(st) == expect
    return new.cpu().numpy()


@pytest.mark.parametrize("d,Hkv,in_place,pad", [(128, 8, False, 0), (64, 3, True, 8), (128, 1, True, 16)])
def test_commit_of_accepted_paths(d, Hkv, in_place, pad):
    rng = np.random.default_rng(d + Hkv)
    sizes, ctx = [16, 1, 0, 40, 33, 64, 9], [0, 63, 5, 100, 62, 191, 128]
    b = workloads.random_batch(rng, sizes, 1, 16, 16, depth_cap=20, max_depth=32)
    lens, path, _ = oracle.accept_batch(b)
    for r, n in enumerate(sizes):  # deeper paths than the walk finds: to a random node
        if n and r != 1:
            j, p = int(rng.integers(0, n)), []
            while j >= 0:
                p.append(j)
                j = int(b.parent[b.node_offsets[r] + j])
            lens[r] = len(p)
            path[r] = -1
            path[r, :len(p)] = p[::-1]
    c = Cache(rng, b.B, 4, Hkv, d)
    ((kt, kv), (vt, vv)), stride = strided(rng, b.T, [Hkv * d, Hkv * d], pad)
    new = commit(c, b, ctx, lens, path, kt, vt, stride, in_place)
    assert np.array_equal(new, np.asarray(ctx) + lens)
    assert lens.max() > 3
    for r in range(b.B):
        for m in range(lens[r]):
            t = b.node_offsets[r] + path[r, m]
            c.put(r, ctx[r] + m, kv[t].reshape(Hkv, d), vv[t].reshape(Hkv, d))
    assert np.array_equal(c.fetch(), c.host)


def test_commit_of_malformed_requests_changes_nothing():
    import tree_speculative_verify_tv_gb300 as tv
    rng = np.random.default_rng(12)
    b = workloads.random_batch(rng, [6, 6, 6], 1, 16, 16, depth_cap=4, max_depth=4)
    c = Cache(rng, 3, 2, 2, 64)
    ((kt, kv), (vt, vv)), stride = strided(rng, b.T, [128, 128], 0)
    good = np.full((3, 4), -1, np.int32)
    good[:, 0] = 0
    one = np.ones(3, np.int32)
    before = c.fetch()

    def bad(expect, ctx=(0, 0, 0), lens=one, path=good, table=None, offsets=None):
        import dataclasses
        bb = b if offsets is None else dataclasses.replace(b, node_offsets=np.asarray(offsets, np.int32))
        c.dev.copy_(cu(before))
        new = commit(c, bb, ctx, np.asarray(lens, np.int32), path, kt, vt, stride, table=table,
                     expect=expect)
        now = c.fetch()
        for r in (0, 2):  # request 1 is the bad one
            assert new[r] == ctx[r] + 1
            assert not np.array_equal(now[c.table[r, 0]], before[c.table[r, 0]])
        assert new[1] == ctx[1]
        assert np.array_equal(now[c.table[1]], before[c.table[1]])

    p = good.copy()
    p[1, 0] = 6
    bad(tv.TV_ERR_TREE, path=p)
    p = good.copy()
    p[1, 0] = -1
    bad(tv.TV_ERR_TREE, path=p)
    bad(tv.TV_ERR_TREE, lens=[1, 5, 1])
    bad(tv.TV_ERR_TREE, lens=[1, -1, 1])
    bad(tv.TV_ERR_SHAPE, ctx=(0, 128, 0))
    bad(tv.TV_ERR_SHAPE, ctx=(0, -1, 0))
    bad(tv.TV_ERR_SHAPE, ctx=(0, 2 ** 31 - 1, 0))
    t = c.table.copy()
    t[1] = c.pages
    bad(tv.TV_ERR_SHAPE, table=t)


# ---------------------------------------------------------------- attention


def check_rows(got, offs, parent, q, K, V, ctx, kt, vt, scale, window, sinks, half):
    want, smax, vmax, n = oracle.qcache_attention(offs, parent, q, K, V, ctx, kt, vt, scale, window,
                                                  sinks, bounds=True)
    d = q.shape[-1]
    e = (d / 16 + 6) * 2 * U * smax + 8 * U
    tol = (vmax * 2 * (e + 2.0 ** -16 + (n / 16 + 16) * U))[..., None] + \
        np.abs(want) * (2.0 ** -8 if half else 2.0 ** -24)
    assert np.isfinite(got).all()
    worst = float((np.abs(got - want) / tol).max()) if got.size else 0.0
    assert worst <= 1, "error %.3g of the bound" % worst
    return worst


def attend(c, b, ctx, H, window=0, sinks=0, half=False, pad=0, seed=0, spike=0.0, table=None,
           parent=None, dctx=None, offsets=None, stream=None, rows=None):
    """(status, outputs, arguments of check_rows)"""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    rng = np.random.default_rng(seed)
    d, Hkv = c.d, c.Hkv
    if rows is None:
        rows = strided(rng, b.T, [H * d, Hkv * d, Hkv * d], pad)
    ((q, qv), (kt, kv), (vt, vv)), stride = rows
    out = torch.full((max(b.T, 1), H, d), float("nan"), device="cuda",
                     dtype=torch.bfloat16 if half else torch.float32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    wsb = tv.tv_qcache_attention_workspace_bytes(b.B, b.T, b.max_nodes, H, Hkv, d, c.mp)
    ws = torch.full((max(wsb, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    scale = d ** -0.5
    par = b.parent if parent is None else parent
    tv.tv_qcache_attention(b.B, b.T, b.max_nodes, H, Hkv, d, c.pages, c.mp,
                           cu(b.node_offsets if offsets is None else offsets),
                           cu(par if b.T else np.zeros(1, np.int32)),
                           cu(np.asarray(ctx if dctx is None else dctx, np.int32)),
                           c.dev_table if table is None else cu(table), window, sinks, q, stride,
                           c.dev, kt, vt, stride, scale, tv.TV_BF16 if half else tv.TV_F32, out, ws,
                           wsb, st, stream=stream)
    s = status(st)
    got = out[:b.T].float().cpu().numpy().astype(np.float64)
    K, V = c.values()
    f = lambda x, h: x.reshape(b.T, h, d).astype(np.float64)  # noqa: E731
    return s, got, (b.node_offsets, b.parent, f(qv, H), K, V, ctx, f(kv, Hkv), f(vv, Hkv), scale,
                    window, sinks, half)


def make(seed, sizes, Hkv, d, ctx, mp=None, depth_cap=10, garbage=True):
    """A cache whose visible positions hold normal rows and the rest 0xFF (scales that say
    NaN) or random bytes, and a batch of trees."""
    rng = np.random.default_rng(seed)
    b = workloads.random_batch(rng, sizes, 1, 16, 16, depth_cap=depth_cap, max_depth=32)
    mp = mp or max(1, -(-max(max(ctx), 1) // 64))
    c = Cache(rng, len(sizes), mp, Hkv, d, fill=0xFF if garbage else None)
    fill(c, rng, ctx)
    return b, c


def fill(c, rng, ctx, v=None):
    """Visible positions with normal rows (in the device's cache by tv_qcache_write; the host
    copy from the device, so that large caches stay quick: the bytes are tested above)."""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    ctx = np.asarray(ctx, np.int32)
    offs = np.concatenate([[0], np.cumsum(ctx)]).astype(np.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = c.Hkv * c.d
    k, _ = bf(rng.normal(size=(max(int(ctx.sum()), 1), w)))
    v, _ = bf(rng.normal(size=(max(int(ctx.sum()), 1), w)))
    tv.tv_qcache_write(c.B, int(ctx.sum()), c.Hkv, c.d, c.pages, c.mp, cu(offs), cu(0 * ctx),
                       c.dev_table, k, v, w, c.dev, st)
    assert status(st) == 0
    c.host = c.fetch()


@pytest.mark.parametrize("H,Hkv,d,half,pad", [
    (4, 4, 64, False, 0), (16, 2, 128, True, 8), (6, 2, 64, True, 0), (8, 1, 128, False, 0),
    (64, 1, 64, False, 16), (96, 1, 128, True, 0), (5, 1, 128, False, 0), (24, 8, 128, True, 0),
])
def test_attention_over_ragged_contexts_and_trees(H, Hkv, d, half, pad):
    ctx = [0, 1, 63, 64, 65, 127, 128, 129, 300]
    b, c = make(H + d, [3, 1, 9, 0, 33, 16, 1, 5, 64], Hkv, d, ctx)
    s, got, args = attend(c, b, ctx, H, half=half, pad=pad, seed=H)
    assert s == 0
    check_rows(got, *args)


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (7, 4), (64, 0), (65, 70), (100, 4), (130, 64),
                                          (500, 3), (4096, 4), (3, 1000)])
def test_window_and_sinks(window, sinks):
    ctx = [0, 2, 64, 150, 321, 640]
    b, c = make(window, [20, 12, 5, 30, 64, 1], 2, 64 if window % 2 else 128, ctx, depth_cap=12)
    s, got, args = attend(c, b, ctx, 8, window=window, sinks=sinks, half=window > 99, seed=window)
    assert s == 0
    check_rows(got, *args)


def test_pages_out_of_the_window_are_not_read():
    import tree_speculative_verify_tv_gb300 as tv
    ctx, W, S = [700, 90], 100, 4
    b, c = make(31, [10, 10], 2, 128, ctx)
    gone = c.table.copy()
    gone[0, 1:9] = [-1, 2 ** 31 - 1, -2 ** 31, c.pages, -1, -1, -1, -1]  # positions 64 .. 575
    s, got, args = attend(c, b, ctx, 4, window=W, sinks=S, table=gone, seed=1)
    assert s == 0
    check_rows(got, *args)
    gone[0, 9] = -1  # 576 .. 639: the window starts at 601
    s, got, _ = attend(c, b, ctx, 4, window=W, sinks=S, table=gone, seed=1)
    assert s == tv.TV_ERR_SHAPE
    assert np.all(got[:10] == 0)
    check_rows(got[10:], np.array([0, 10]), b.parent[10:], args[2][10:], args[3][1:],
               args[4][1:], ctx[1:], args[6][10:], args[7][10:], *args[8:])


def test_256_node_trees():
    ctx = [400, 0, 77]
    b, c = make(41, [256, 130, 200], 1, 128, ctx, depth_cap=32)
    s, got, args = attend(c, b, ctx, 4, seed=5)
    assert s == 0
    check_rows(got, *args)


def test_a_chain_of_256_nodes_with_a_window():
    ctx = [90]
    b, c = make(42, [256], 2, 64, ctx)
    b.parent[:] = np.arange(-1, 255, dtype=np.int32)
    s, got, args = attend(c, b, ctx, 4, window=100, sinks=3, seed=6)
    assert s == 0
    check_rows(got, *args)


@pytest.mark.parametrize("B", [1, 300])
def test_long_and_many_contexts(B):
    # one context over the whole GPU, and more requests than SMs with one token each
    rng = np.random.default_rng(B)
    ctx = [20000] if B == 1 else rng.integers(0, 200, B).tolist()
    b, c = make(B, [5] if B == 1 else [1] * B, 1 if B == 1 else 2, 128, ctx)
    s, got, args = attend(c, b, ctx, 4, seed=B, half=B > 1)
    assert s == 0
    check_rows(got, *args)


def test_scores_that_jump_between_tiles():
    # keys along the queries with growing length: the running maximum rises again and again
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    d, L = 128, 1500
    b, c = make(51, [6], 1, d, [L], garbage=False)
    rng = np.random.default_rng(52)
    rows = strided(rng, b.T, [4 * d, d, d], 0)
    u = rows[0][0][1].reshape(-1, d)[0]
    k = rng.normal(size=(L, d))
    for i, pos in enumerate(range(10, L, 150)):
        k[pos] = u / np.linalg.norm(u) * np.sqrt(d) * (4 + 5 * i)
    write(c, rng, [L], [0], k=k, v=rng.normal(size=(L, d)))
    s, got, args = attend(c, b, [L], 4, rows=rows)
    assert s == 0
    check_rows(got, *args)


def test_malformed_requests_give_zero_rows():
    import tree_speculative_verify_tv_gb300 as tv
    ctx = [100, 70, 128]
    b, c = make(61, [4, 20, 6], 2, 64, ctx, mp=2)
    s0, good, args = attend(c, b, ctx, 4, seed=3)
    assert s0 == 0
    check_rows(good, *args)
    first, last = slice(0, 4), slice(24, 30)

    def only_middle_zero(got):
        assert np.array_equal(got[first], good[first]) and np.array_equal(got[last], good[last])
        assert np.all(got[4:24] == 0)

    for at, p in ((4 + 3, 3), (4 + 5, 6), (4 + 1, -2), (4, 2 ** 31 - 1), (4 + 19, -2 ** 31)):
        par = b.parent.copy()
        par[at] = p
        s, got, _ = attend(c, b, ctx, 4, seed=3, parent=par)
        assert s == tv.TV_ERR_TREE
        only_middle_zero(got)
    for bad in (-1, 129, 2 ** 31 - 1, -2 ** 31):
        s, got, _ = attend(c, b, ctx, 4, seed=3, dctx=[100, bad, 128])
        assert s == tv.TV_ERR_SHAPE
        only_middle_zero(got)
    for page in (-1, c.pages, 2 ** 31 - 1):
        t = c.table.copy()
        t[1, 1] = page
        s, got, _ = attend(c, b, ctx, 4, seed=3, table=t)
        assert s == tv.TV_ERR_SHAPE
        only_middle_zero(got)
    for offs in ([0, 4, 31, 30], [0, 4, -1, 30]):
        s, got, _ = attend(c, b, ctx, 4, seed=3, offsets=np.array(offs, np.int32))
        assert s == tv.TV_ERR_TREE
        assert np.array_equal(got[first], good[first])


def test_not_a_number_stays_in_its_row():
    # a NaN query: its own row only
    import torch
    ctx = [200]
    b, c = make(71, [5], 1, 128, ctx)
    rng = np.random.default_rng(72)
    rows = strided(rng, b.T, [2 * 128, 128, 128], 0)
    _, good, _ = attend(c, b, ctx, 2, rows=rows)
    rows[0][0][0][3, 128 + 9] = float("nan")
    s, got, _ = attend(c, b, ctx, 2, rows=rows)
    assert s == 0
    assert np.isnan(got[3, 1]).all()
    keep = np.ones((5, 2), bool)
    keep[3, 1] = False
    assert np.array_equal(got[keep], good[keep])


def test_repeats_are_equal_bit_for_bit_and_other_streams_serve():
    import torch
    ctx = [1000, 33]
    b, c = make(81, [12, 3], 2, 128, ctx)
    _, first, _ = attend(c, b, ctx, 8, seed=2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, None, side):
        s, got, _ = attend(c, b, ctx, 8, seed=2, stream=stream)
        assert s == 0 and np.array_equal(got, first)


def test_two_decode_steps_in_a_graph():
    """accept -> commit in place -> attention over the grown cache, captured once and
    replayed: the second replay attends to what the first one committed."""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    rng = np.random.default_rng(91)
    Hkv, H, d, ctx0 = 2, 8, 64, [60, 10, 127]
    b, c = make(92, [9, 4, 16], Hkv, d, ctx0, mp=4, depth_cap=5)
    ((q, qv), (kt, kv), (vt, vv)), stride = strided(rng, b.T, [H * d, Hkv * d, Hkv * d], 0)
    ctx, offs, par = cu(np.array(ctx0, np.int32)), cu(b.node_offsets), cu(b.parent)
    draft, target, root = cu(b.draft), cu(b.target), cu(b.root_argmax)
    ln, bonus = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    path = torch.zeros((3, b.max_depth), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros((b.T, H, d), dtype=torch.float32, device="cuda")
    wsb = tv.tv_qcache_attention_workspace_bytes(3, b.T, b.max_nodes, H, Hkv, d, c.mp)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device="cuda")

    def step():
        tv.tv_accept_greedy(3, b.T, b.max_nodes, b.max_depth, offs, par, draft, target, root, ln,
                            path, bonus, st)
        tv.tv_qcache_commit(3, b.T, b.max_nodes, b.max_depth, Hkv, d, c.pages, c.mp, offs, path, ln,
                            ctx, c.dev_table, kt, vt, stride, c.dev, ctx, st)
        tv.tv_qcache_attention(3, b.T, b.max_nodes, H, Hkv, d, c.pages, c.mp, offs, par, ctx,
                               c.dev_table, 0, 0, q, stride, c.dev, kt, vt, stride, 0.125,
                               tv.TV_F32, out, ws, wsb, st)

    step()  # loads the kernels before the capture
    torch.cuda.synchronize()
    ctx.copy_(cu(np.array(ctx0, np.int32)))
    c.dev.copy_(cu(c.host))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    lens, p, _ = oracle.accept_batch(b)
    now = list(ctx0)
    for _ in range(2):
        g.replay()
        assert status(st) == 0
        for r in range(3):
            for m in range(lens[r]):
                t = b.node_offsets[r] + p[r, m]
                c.put(r, now[r] + m, kv[t].reshape(Hkv, d), vv[t].reshape(Hkv, d))
            now[r] += int(lens[r])
        assert ctx.cpu().numpy().tolist() == now
        assert np.array_equal(c.fetch(), c.host)
        K, V = c.values()
        f = lambda x, h: x.reshape(b.T, h, d).astype(np.float64)  # noqa: E731
        check_rows(out.cpu().numpy().astype(np.float64), b.node_offsets, b.parent, f(qv, H), K, V, now,
                   f(kv, Hkv), f(vv, Hkv), 0.125, 0, 0, False)
    assert lens.max() > 0
