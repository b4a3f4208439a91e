"""The operators around int8 experts on the GPU, against their 64-bit references
(int8_ops_ref): scored routing, int8 products, the int8-activation FFN, the block
norms, and a decoder layer's run of them, eager and from a CUDA graph."""
import numpy as np
import pytest
import torch

import int8_ops_ref as ref
import moe_router_softmax_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def bf16(a):
    """(device bf16, its value in fp64) of a float array."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16()
    return t.to(DEV), t.double().numpy()


def f64(t):
    return t.double().cpu().numpy()


def no_device_error():
    assert moe.moe_take_device_errors() == (0, 0)


# ------------------------------------------------------------------ routing

def check_route(lg, k, bias=None, score="softmax", **kw):
    sc = {"softmax": moe.MOE_SCORE_SOFTMAX, "sigmoid": moe.MOE_SCORE_SIGMOID}[score]
    ids, w = moe.moe_route_scored(dev(lg), k, bias=None if bias is None else dev(bias), score=sc, **kw)
    rid, rw = ref.route(lg, k, bias=bias, score=score, **kw)
    assert np.array_equal(ids.cpu().numpy(), rid)
    # rounded once to fp32 (half a step, or of the smallest subnormal), after fp64 sums whose own error is far below it
    assert np.all(np.abs(f64(w) - rw) <= (1 + 1e-6) * ref.U32 * np.abs(rw) + 2.0 ** -149)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (3, 33, 5), (5, 64, 32), (2, 200, 7), (17, 256, 8),
                                   (2, 500, 4), (3, 1000, 32), (2, 1024, 1), (129, 96, 6)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scored(T, E, k, score):
    r = np.random.default_rng([T, E, k])
    lg = (2 * r.standard_normal((T, E))).astype(np.float32)
    b = (0.1 * r.standard_normal(E)).astype(np.float32)
    check_route(lg, k, score=score)
    check_route(lg, k, bias=b, score=score, renorm=False, scale=2.5)
    check_route(lg, k, bias=10 * b, score=score)  # a bias that outweighs the scores


@pytest.mark.parametrize("T,E,G,tg,gt,k", [
    (1, 256, 8, 4, 2, 8), (9, 256, 8, 4, 1, 8), (3, 160, 8, 3, 2, 6), (4, 165, 5, 3, 1, 6), (2, 66, 22, 3, 2, 6),
    (2, 1024, 32, 7, 2, 32), (3, 96, 3, 1, 2, 32), (5, 64, 32, 32, 2, 32), (2, 30, 30, 4, 1, 4), (1, 1000, 8, 2, 2, 9),
    (3, 68, 17, 5, 2, 20), (2, 12, 6, 6, 1, 12)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scored_groups(T, E, G, tg, gt, k, score):
    r = np.random.default_rng([T, E, G])
    lg = (2 * r.standard_normal((T, E))).astype(np.float32)
    b = (0.1 * r.standard_normal(E)).astype(np.float32)
    for bias in (None, b):
        check_route(lg, k, bias=bias, score=score, n_group=G, topk_group=tg, group_top=gt)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G", [1, 4])
def test_route_scored_masks_and_ties(score, G):
    low, E, k = ref.LOWEST, 32, 6
    r = np.random.default_rng(3)
    lg = r.standard_normal((12, E)).astype(np.float32)
    lg[0] = 0.0                                   # all equal
    lg[1] = -np.inf                               # nothing left
    lg[2] = np.nan
    lg[3] = low
    lg[4, 3:] = -np.inf                           # fewer live than k
    lg[5, ::2] = np.nan
    lg[6, 5] = np.inf
    lg[7, 5] = lg[7, 9] = np.inf                  # two of them
    lg[8] = np.repeat(lg[8, ::4], 4)              # ties in runs
    lg[9, 8:16] = low                             # a whole group of four
    lg[10] = -200.0 - np.arange(E)                # tiny scores
    lg[11] = np.where(np.arange(E) % 3 == 0, -0.0, 0.0)
    kw = dict(score=score, n_group=G, topk_group=min(G, 2), group_top=1 + (G > 1))
    check_route(lg, k, **kw)
    b = np.zeros(E, np.float32)
    b[[0, 9, 17]] = [-np.inf, np.nan, low]
    check_route(lg, k, bias=b, **kw)
    check_route(lg, k, bias=b, renorm=False, **kw)
    check_route(lg, k, bias=np.full(E, -np.inf, np.float32), **kw)


@pytest.mark.parametrize("E,k,G,tg", [(64, 3, 4, 2), (40, 32, 1, 1), (128, 8, 1, 1), (96, 11, 3, 2)])
def test_route_scored_many_tokens(E, k, G, tg):
    """Batches in which a warp takes several tokens, ties and masks among them."""
    T = 6001
    r = np.random.default_rng(E)
    lg = (2 * r.standard_normal((T, E))).astype(np.float32)
    lg[::7] = np.round(lg[::7])
    lg[::11, : E // 2] = -np.inf
    lg[::501] = -np.inf
    b = (0.1 * r.standard_normal(E)).astype(np.float32)
    check_route(lg, k, bias=b, score="sigmoid", n_group=G, topk_group=tg, group_top=1 + (G > 1))
    check_route(lg, k, renorm=False, n_group=G, topk_group=tg)


def test_route_scored_decides_in_64_bits():
    """Choices nearer to one another than fp32 tells apart."""
    E = 64
    lg = np.zeros((2, E), np.float32)
    b = np.zeros(E, np.float32)
    lg[:, 40], lg[:, 7] = 1.0, np.nextafter(np.float32(1.0), np.float32(2.0))
    lg[1, 7] = np.nextafter(np.float32(1.0), np.float32(0.0))
    for score in ("softmax", "sigmoid"):
        check_route(lg, 2, bias=b, score=score)
        check_route(lg, 2, bias=b + np.float32(1000.0), score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scored_with_biases_that_cancel(score):
    """Group scores that are small sums of large choices, and biases of every size."""
    T, E = 400, 64
    r = np.random.default_rng(17)
    lg = (2 * r.standard_normal((T, E))).astype(np.float32)
    b = np.zeros(E, np.float32)
    b[0::8], b[1::8] = 3e4, -3e4
    check_route(lg, 6, bias=b, score=score, n_group=8, topk_group=3, group_top=2)
    b = (10.0 ** r.uniform(-6, 6, E) * np.where(r.random(E) < 0.5, -1, 1)).astype(np.float32)
    for G in (1, 4, 8):
        check_route(lg, 6, bias=b, score=score, n_group=G, topk_group=max(G // 2, 1), group_top=1 + (G > 1))
    b = np.full(E, 3e38, np.float32)
    b[E // 2:] = -3e38
    check_route(lg, 6, bias=b, score=score, n_group=8, topk_group=5, group_top=2)


def test_route_scored_feeds_the_permute():
    T, E, k = 21, 48, 4
    r = np.random.default_rng(5)
    lg = r.standard_normal((T, E)).astype(np.float32)
    lg[4] = -np.inf
    lg[6, 2:] = -np.inf
    ids, w = moe.moe_route_scored(dev(lg), k)
    counts, offsets, sr, rp = (t.cpu().numpy() for t in moe.moe_permute(ids, E))
    flat = ids.cpu().numpy().ravel()
    assert counts.tolist() == [int((flat == e).sum()) for e in range(E)]
    assert np.array_equal(rp < 0, flat < 0) and (rp[4 * k:5 * k] == -1).all()


# ------------------------------------------------------------------ int8 product

def random_codes(r, *shape, full=False):
    q = r.integers(-128 if full else -127, 128, shape, dtype=np.int64).astype(np.int8)
    return q


@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 16, 31, 64, 65, 130, 257])
@pytest.mark.parametrize("N,K", [(1, 16), (7, 64), (33, 80), (128, 128), (130, 272), (300, 1040), (64, 2816), (129, 528),
                                 (2500, 544), (5000, 1040), (9473, 400)])
def test_linear_int8(T, N, K):
    r = np.random.default_rng([T, N, K])
    xq, wq = random_codes(r, T, K, full=True), random_codes(r, N, K, full=True)
    sx = (0.01 + r.random(T)).astype(np.float32)
    sw = ((0.01 + r.random(N)) * np.where(r.random(N) < 0.5, -1, 1)).astype(np.float32)
    y = ref.linear(xq, sx, wq, sw)
    a = [dev(v) for v in (xq, sx, wq, sw)]
    out = moe.moe_linear_int8(*a, dtype=torch.float32)
    # the exact sum: one rounding to fp32 and two products, half a step each
    assert np.all(np.abs(f64(out) - y) <= 3 * (1 + 1e-6) * ref.U32 * np.abs(y))
    out = moe.moe_linear_int8(*a)
    assert np.all(np.abs(f64(out) - y) <= (ref.UBF * (1 + 3 * ref.U32) + 3 * ref.U32) * (1 + 1e-6) * np.abs(y))
    no_device_error()


@pytest.mark.parametrize("T,N,K", [(256, 18944, 128), (257, 18944, 144), (300, 9601, 272), (2000, 2433, 1040),
                                   (515, 6400, 2816), (4097, 1100, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_int8_large(T, N, K, dtype):
    """Products that fill the GPU (the exact sums in fp64 on the device)."""
    g = torch.Generator(DEV).manual_seed(T)
    xq = torch.randint(-128, 128, (T, K), generator=g, dtype=torch.int8, device=DEV)
    wq = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8, device=DEV)
    sx, sw = 0.1 + torch.rand(T, generator=g, device=DEV), 0.1 + torch.rand(N, generator=g, device=DEV)
    y = (xq.double() @ wq.double().t()) * sx.double()[:, None] * sw.double()
    out = moe.moe_linear_int8(xq, sx, wq, sw, dtype=dtype).double()
    rel = 3 * ref.U32 if dtype is torch.float32 else ref.UBF * (1 + 3 * ref.U32) + 3 * ref.U32
    assert bool(((out - y).abs() <= rel * (1 + 1e-6) * y.abs()).all())
    no_device_error()


@pytest.mark.parametrize("T", [1, 4, 40])
def test_linear_int8_extreme_sums(T):
    """The largest sums int32 has to hold, and rows of zero codes and scales."""
    K, N = 65536, 40
    xq = np.full((T, K), -128, np.int8)
    wq = np.full((N, K), -128, np.int8)
    wq[1::2] = 127
    wq[5] = 0
    sx, sw = np.ones(T, np.float32), np.ones(N, np.float32)
    sx[0], sw[3] = 0.0, 0.0
    y = ref.linear(xq, sx, wq, sw)
    out = moe.moe_linear_int8(dev(xq), dev(sx), dev(wq), dev(sw), dtype=torch.float32)
    assert np.all(np.abs(f64(out) - y) <= 3 * (1 + 1e-6) * ref.U32 * np.abs(y))


@pytest.mark.parametrize("T", [3, 70])
def test_linear_int8_leaves_the_rest(T):
    """Rows and columns around an output that lies inside a larger buffer."""
    N, K = 37, 96
    r = np.random.default_rng(T)
    a = [dev(v) for v in (random_codes(r, T, K), np.ones(T, np.float32), random_codes(r, N, K), np.ones(N, np.float32))]
    buf = torch.full(((T * N + 15) // 8 * 8 + 64,), 7.0, device=DEV)
    y = buf[32:32 + T * N].view(T, N)
    moe.moe_linear_int8(*a, y=y)
    assert torch.equal(y, moe.moe_linear_int8(*a, dtype=torch.float32))
    assert (buf[:32] == 7).all() and (buf[32 + T * N:] == 7).all()


# ------------------------------------------------------------------ FFN with int8 activations

def int8_layer(E, H, I, seed, slots=None, missing=()):
    """Layer with random codes; its pieces on the host.  `slots`: slot table."""
    r = np.random.default_rng(seed)
    q13, q2 = random_codes(r, E, 2 * I, H), random_codes(r, E, H, I)
    s13 = (0.002 * (0.5 + r.random((E, 2 * I)))).astype(np.float32)
    s2 = (0.002 * (0.5 + r.random((E, H)))).astype(np.float32)
    eb = (moe.moe_expert_bytes(moe.MOE_W_INT8, H, I) + 255) // 256 * 256
    blobs = np.zeros((E, eb), np.uint8)
    for e in range(E):
        b = np.concatenate([v[e].view(np.uint8).ravel() for v in (q13, s13, q2, s2)])
        blobs[e, :b.size] = b
    home = blobs.copy()
    pool = table = None
    if slots is not None:
        pool = np.zeros((max(slots) + 1, eb), np.uint8)
        for e, s in enumerate(slots):
            if s >= 0:
                pool[s] = blobs[e]
                home[e] = 0xA5
        pool, table = dev(pool.ravel()), dev(np.array(slots, np.int32))
    L = moe.MoeLayer(moe.MOE_W_INT8, E, H, I, dev(home.ravel()), pool=pool, slot_table=table, expert_bytes=eb)
    return L, (q13, s13, q2, s2)


def tokens(T, H, seed):
    r = np.random.default_rng([seed, T, H])
    q, s = ref.codes(r.standard_normal((T, H)) * np.exp(0.5 * r.standard_normal((T, 1))))
    return q.astype(np.int8), s.astype(np.float32)


def check_ffn(L, pieces, xq, sx, ids, rows, rp, only=None):
    T, k = ids.shape
    rows, rp = f64(rows), rp.cpu().numpy()
    q13, s13, q2, s2 = pieces
    for t in range(T):
        if only is not None and t not in only:
            continue
        for j in range(k):
            e, p = ids[t, j], rp[t * k + j]
            if e < 0 or e >= L.E:
                assert p == -1
                continue
            row, tol = ref.ffn_row(xq[t], sx[t], q13[e], s13[e], q2[e], s2[e])
            assert np.all(np.abs(rows[p] - row) <= tol), (t, j, float((np.abs(rows[p] - row) - tol).max()))


@pytest.mark.parametrize("E,H,I,k", [(8, 256, 128, 2), (5, 64, 64, 1), (16, 320, 192, 4), (12, 128, 704, 3)])
@pytest.mark.parametrize("T", [1, 2, 3, 7, 20, 65, 150])
def test_ffn_w8a8(E, H, I, k, T):
    L, pieces = int8_layer(E, H, I, seed=E + H)
    xq, sx = tokens(T, H, seed=k)
    r = np.random.default_rng([T, E])
    ids = np.argsort(r.standard_normal((T, E)) + 0.7 * r.standard_normal(E), axis=1)[:, :k].astype(np.int32)
    if T > 2:
        ids[1, 0] = -1          # a dropped route
        ids[2, k - 1] = E + 3   # an id that is none
        xq[0], sx[0] = 0, 0.0   # a token of zeros
    counts, offsets, sr, rp = moe.moe_permute(dev(ids), E)
    rows = torch.full((T * k, H), float("nan"), device=DEV)
    moe.moe_grouped_ffn_w8a8(L, dev(xq), dev(sx), k, counts, offsets, sr, rows=rows)
    check_ffn(L, pieces, xq, sx, ids, rows, rp)
    n = int(offsets[-1])
    assert torch.isnan(rows[n:]).all() and torch.isfinite(rows[:n]).all()  # rows behind the last route: untouched
    again = moe.moe_grouped_ffn_w8a8(L, dev(xq), dev(sx), k, counts, offsets, sr)
    assert torch.equal(again[:n], rows[:n])
    no_device_error()


@pytest.mark.parametrize("T", [1, 4, 64, 300])
def test_ffn_w8a8_repository_shape(T):
    """128 experts, hidden 2816, intermediate 704, top-8; a few tokens checked in full."""
    E, H, I, k = 128, 2816, 704, 8
    L, pieces = int8_layer(E, H, I, seed=1)
    xq, sx = tokens(T, H, seed=2)
    ids, w = moe.moe_route_scored(torch.randn((T, E), device=DEV, generator=torch.Generator(DEV).manual_seed(T)), k)
    counts, offsets, sr, rp = moe.moe_permute(ids, E)
    rows = moe.moe_grouped_ffn_w8a8(L, dev(xq), dev(sx), k, counts, offsets, sr)
    check_ffn(L, pieces, xq, sx, ids.cpu().numpy(), rows, rp, only={0, T // 2, T - 1})
    no_device_error()


@pytest.mark.parametrize("T", [1, 3, 80])
def test_ffn_w8a8_every_token_to_one_expert(T):
    E, H, I = 6, 192, 128
    L, pieces = int8_layer(E, H, I, seed=9)
    xq, sx = tokens(T, H, seed=3)
    ids = np.full((T, 1), 4, np.int32)
    counts, offsets, sr, rp = moe.moe_permute(dev(ids), E)
    rows = moe.moe_grouped_ffn_w8a8(L, dev(xq), dev(sx), 1, counts, offsets, sr)
    check_ffn(L, pieces, xq, sx, ids, rows, rp)
    # no route at all
    counts, offsets, sr, rp = moe.moe_permute(dev(np.full((T, 1), -1, np.int32)), E)
    rows.fill_(3.0)
    moe.moe_grouped_ffn_w8a8(L, dev(xq), dev(sx), 1, counts, offsets, sr, rows=rows)
    assert (rows == 3.0).all()
    no_device_error()


@pytest.mark.parametrize("E,H,I,k,T,skew", [
    (2, 128, 64, 1, 600, 0.9),       # an expert with more routes than one block holds
    (3, 192, 128, 2, 700, 0.0),
    (300, 64, 64, 5, 333, 0.0),      # more experts than lanes or warps
    (1024, 64, 64, 3, 900, 0.5), (40, 128, 128, 8, 257, 0.7)])
def test_ffn_w8a8_many_routes(E, H, I, k, T, skew):
    L, pieces = int8_layer(E, H, I, seed=E)
    xq, sx = tokens(T, H, seed=5)
    r = np.random.default_rng([E, T])
    score = r.standard_normal((T, E))
    score[r.random(T) < skew, 0] -= 100.0   # that share of the tokens takes expert 0
    ids = np.argsort(score, axis=1)[:, :k].astype(np.int32)
    counts, offsets, sr, rp = moe.moe_permute(dev(ids), E)
    rows = moe.moe_grouped_ffn_w8a8(L, dev(xq), dev(sx), k, counts, offsets, sr)
    check_ffn(L, pieces, xq, sx, ids, rows, rp)
    no_device_error()


def test_ffn_w8a8_the_same_expert_twice():
    """A token that names an expert twice has two routes of it, with equal rows."""
    E, H, I, k = 4, 128, 64, 2
    L, pieces = int8_layer(E, H, I, seed=8)
    for T in (1, 300):
        xq, sx = tokens(T, H, seed=T)
        ids = np.full((T, k), 2, np.int32)
        counts, offsets, sr, rp = moe.moe_permute(dev(ids), E)
        rows = moe.moe_grouped_ffn_w8a8(L, dev(xq), dev(sx), k, counts, offsets, sr)
        check_ffn(L, pieces, xq, sx, ids, rows, rp, only={0, T - 1})
        by_route = rows[rp.long()].view(T, k, H)
        assert torch.equal(by_route[:, 0], by_route[:, 1])
    no_device_error()


@pytest.mark.parametrize("T", [1, 5, 70])
def test_ffn_w8a8_slot_table(T):
    E, H, I, k = 8, 256, 128, 3
    slots = [-1, 11, 0, -1, 5, 7, -1, 2]
    L, pieces = int8_layer(E, H, I, seed=4, slots=slots)
    xq, sx = tokens(T, H, seed=6)
    r = np.random.default_rng(T)
    ids = np.argsort(r.random((T, E)), axis=1)[:, :k].astype(np.int32)
    counts, offsets, sr, rp = moe.moe_permute(dev(ids), E)
    rows = moe.moe_grouped_ffn_w8a8(L, dev(xq), dev(sx), k, counts, offsets, sr)
    check_ffn(L, pieces, xq, sx, ids, rows, rp)
    no_device_error()
    # a slot past the pool: refused, reported, the other rows as before
    L.slot_table[4] = L.pool_slots
    out = torch.full_like(rows, float("nan"))
    moe.moe_grouped_ffn_w8a8(L, dev(xq), dev(sx), k, counts, offsets, sr, rows=out)
    bad = np.zeros(T * k, bool)
    bad[rp.cpu().numpy()[ids.ravel() == 4]] = True
    bad = torch.from_numpy(bad).to(DEV)
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], rows[~bad])
    code, info = moe.moe_take_device_errors()
    assert (code != 0 and info == L.pool_slots) if bool(bad.any()) else code == 0


def test_ffn_w8a8_empty_batch():
    L, _ = int8_layer(4, 64, 64, seed=0)
    z = lambda *s, d=torch.int32: torch.zeros(s, dtype=d, device=DEV)  # noqa: E731
    rows = moe.moe_grouped_ffn_w8a8(L, z(0, 64, d=torch.int8), z(0, d=torch.float32), 2, z(4), z(5), z(0))
    assert rows.shape == (0, 64)


# ------------------------------------------------------------------ norms

def check_next(out, y_stored, nw, eps, off):
    n, rel = ref.norm(y_stored, nw, eps, off)
    if out.xn is not None:
        assert np.all(np.abs(f64(out.xn) - n) <= (ref.UBF * (1 + rel) + rel) * np.abs(n) + 2.0 ** -134)
    if out.xq is not None:
        _, s = ref.codes(n)
        assert np.all(np.abs(f64(out.sx) - s) <= (rel + 2 * ref.U32) * s + 2.0 ** -149)
        q = n / np.where(s > 0, s, 1.0)[:, None]
        # the nearest code of a quotient that is off by both errors
        assert np.all(np.abs(f64(out.xq) - q) <= 0.5 + 127 * (2 * rel + 3 * ref.U32))


@pytest.mark.parametrize("T,H", [(1, 64), (3, 128), (2, 320), (5, 2816), (1, 4160), (2, 8192), (1, 8256), (2, 16384),
                                 (300, 192), (33, 1024), (258, 16384), (300, 8256), (257, 4160)])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_norm(T, H, offset):
    r = np.random.default_rng([T, H])
    x = r.standard_normal((T, H)) * np.exp(r.standard_normal((T, 1)))
    x[:, 3] *= 30
    if T > 1:
        x[1] = 0.0
    xt, xv = bf16(x)
    wt, wv = bf16(1.0 + 0.3 * r.standard_normal(H))
    out = moe.moe_norm(xt, wt, eps=1e-5, offset=offset, codes=True)
    check_next(out, xv, wv, 1e-5, offset)
    only = moe.moe_norm(xt, wt, eps=1e-5, offset=offset, codes=True, want_xn=False)
    assert only.xn is None and torch.equal(only.xq, out.xq) and torch.equal(only.sx, out.sx)
    assert torch.equal(moe.moe_norm(xt, wt, eps=1e-5, offset=offset).xn, out.xn)
    if T > 1:
        assert float(out.sx[1]) == 0.0 and (out.xq[1] == 0).all()


@pytest.mark.parametrize("T,H,k", [(257, 2816, 0), (257, 2816, 3), (260, 16384, 0), (258, 8256, 1), (300, 192, 9)])
def test_after_block_many_rows(T, H, k):
    test_after_block(T, H, "all", k)


@pytest.mark.parametrize("T,H", [(1, 64), (3, 192), (4, 2816), (1, 8256), (2, 16384), (70, 256)])
@pytest.mark.parametrize("form", ["plain", "norm", "gates", "all"])
@pytest.mark.parametrize("k", [0, 1, 8, 11, 32])
def test_after_block(T, H, form, k):
    r = np.random.default_rng([T, H, k])
    eps, off, rs, bs = 1e-6, 0.5, 0.75, -1.25
    res, resv = bf16(r.standard_normal((T, H)))
    pw = gh = gt = nw = None
    pv = ghv = gtv = nv = None
    if form in ("norm", "all"):
        pw, pv = bf16(0.3 * r.standard_normal(H))
    if form in ("gates", "all"):
        ghv, gtv = r.standard_normal(H).astype(np.float32), r.standard_normal(T).astype(np.float32)
        gh, gt = dev(ghv), dev(gtv)
    if form in ("norm", "all"):
        nw, nv = bf16(0.3 * r.standard_normal(H))
    kw = dict(post_weight=pw, gate_h=gh, gate_t=gt, next_weight=nw, eps=eps, offset=off, residual_scale=rs,
              block_scale=bs, codes=nw is not None)
    if k == 0:
        z, zv = bf16(r.standard_normal((T, H)))
        mag = np.zeros_like(zv)
        out = moe.moe_residual_norm(z, res, **kw)
    else:
        rows = r.standard_normal((T * k, H)).astype(np.float32)
        pos = r.permutation(T * k).astype(np.int32)
        w = r.random((T, k)).astype(np.float32)
        pos[r.random(T * k) < 0.1] = -1
        if T > 2:
            pos[k:2 * k] = -1            # a token without a route
            pos[2 * k] = T * k + 5       # and a position that is none
        zv, mag = ref.combine(rows, pos, w)
        out = moe.moe_combine_norm(dev(rows), dev(pos), dev(w), res, **kw)
    y, tol = ref.after_block(zv, mag, resv, pv, ghv, gtv, eps, off, rs, bs)
    assert np.all(np.abs(f64(out.y) - y) <= ref.UBF * (np.abs(y) + tol) + tol + 2.0 ** -134)
    if nw is None:
        assert out.xn is None and out.xq is None and out.sx is None
        return
    check_next(out, f64(out.y), nv, eps, off)
    # the same as the two calls, and in place
    two = moe.moe_norm(out.y, nw, eps=eps, offset=off, codes=True)
    assert torch.equal(two.xn, out.xn) and torch.equal(two.xq, out.xq) and torch.equal(two.sx, out.sx)
    if k == 0:
        for tgt in ("residual", "z"):
            a, b = z.clone(), res.clone()
            o = moe.moe_residual_norm(a, b, y=b if tgt == "residual" else a, **kw)
            assert torch.equal(o.y, out.y) and torch.equal(o.xn, out.xn)
    else:
        b = res.clone()
        o = moe.moe_combine_norm(dev(rows), dev(pos), dev(w), b, y=b, **kw)
        assert torch.equal(o.y, out.y) and torch.equal(o.xq, out.xq)


@pytest.mark.parametrize("H", [192, 2816, 8256])
def test_norm_rows_do_not_depend_on_the_batch(H):
    r = np.random.default_rng(H)
    x, _ = bf16(r.standard_normal((300, H)))
    w, _ = bf16(r.standard_normal(H))
    whole = moe.moe_norm(x, w, codes=True)
    for t in (1, 2, 30):
        part = moe.moe_norm(x[:t], w, codes=True)
        assert torch.equal(part.xn, whole.xn[:t]) and torch.equal(part.xq, whole.xq[:t])


def test_norm_with_infinities_and_nan():
    x = torch.ones((4, 128), dtype=torch.bfloat16, device=DEV)
    x[1, 7] = float("nan")
    x[2, 7] = float("inf")
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    out = moe.moe_norm(x, w, codes=True)
    clean = moe.moe_norm(torch.ones((1, 128), dtype=torch.bfloat16, device=DEV), w, codes=True)
    assert torch.isnan(out.xn[1]).all() and (out.xq[1] == 0).all()
    assert torch.isnan(out.xn[2, 7]) and (out.xn[2, :7] == 0).all()
    for t in (0, 3):  # the rows beside them
        assert torch.equal(out.xn[t], clean.xn[0]) and torch.equal(out.xq[t], clean.xq[0])


def test_empty_batches():
    e = lambda *s, d=torch.float32: torch.empty(s, dtype=d, device=DEV)  # noqa: E731
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    x = e(0, 64, d=torch.bfloat16)
    out = moe.moe_norm(x, w, codes=True)
    assert out.xn.shape == out.xq.shape == (0, 64) and out.sx.shape == (0,)
    assert moe.moe_residual_norm(x, x, w, next_weight=w, codes=True).y.shape == (0, 64)
    assert moe.moe_combine_norm(e(0, 64), e(0, d=torch.int32), e(0, 3), x, w, next_weight=w).y.shape == (0, 64)
    assert moe.moe_linear_int8(out.xq, out.sx, torch.ones((8, 64), dtype=torch.int8, device=DEV), e(8)).shape == (0, 8)
    assert moe.moe_route_scored(e(0, 16), 2)[0].shape == (0, 2)


# ------------------------------------------------------------------ refusals of the binding

def test_binding_refusals():
    i8 = torch.zeros((4, 64), dtype=torch.int8, device=DEV)
    s = torch.ones(4, device=DEV)
    with pytest.raises(ValueError, match="shape"):
        moe.moe_linear_int8(i8, s[:3], i8, s)
    with pytest.raises(ValueError, match="shape"):
        moe.moe_linear_int8(i8, s, i8[:, :32].contiguous(), s)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_linear_int8(torch.zeros((64, 4), dtype=torch.int8, device=DEV).t(), s, i8, s)
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_linear_int8(i8, s, i8, s, dtype=torch.float16)
    with pytest.raises(ValueError, match="expected"):
        moe.moe_linear_int8(i8, s.cpu(), i8, s)
    with pytest.raises(moe.MoeError):
        moe.moe_linear_int8(i8.flatten()[8:8 + 64].view(1, 64), s[:1], i8, s)  # 8-byte aligned
    with pytest.raises(ValueError, match="shape"):
        moe.moe_route_scored(torch.zeros((2, 8), device=DEV), 2, bias=torch.zeros(7, device=DEV))
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_route_scored(torch.zeros((2, 8), device=DEV, dtype=torch.bfloat16), 2)
    with pytest.raises(moe.MoeError, match="k=9"):
        moe.moe_route_scored(torch.zeros((2, 8), device=DEV), 9)
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_norm(x, x[0].float())
    with pytest.raises(ValueError, match="shape"):
        moe.moe_residual_norm(x[:1], x)
    with pytest.raises(moe.MoeError, match="eps"):
        moe.moe_norm(x, x[0], eps=0.0)


# ------------------------------------------------------------------ a run of them together

def _decoder(T, E=16, H=256, I=128, k=4, n=3):
    """A chain of n MoE blocks over one residual stream; returns the call and what it writes."""
    g = torch.Generator(DEV).manual_seed(T)
    layers = [int8_layer(E, H, I, seed=20 + l)[0] for l in range(n)]
    rnd = lambda *s: torch.randn(s, device=DEV, generator=g)  # noqa: E731
    pre = [(1 + 0.1 * rnd(H)).bfloat16() for _ in range(n + 1)]
    post = [(1 + 0.1 * rnd(H)).bfloat16() for _ in range(n)]
    qr, sr_ = moe.moe_quantize_int8((0.1 * rnd(E, H)).bfloat16())
    bias = 0.02 * rnd(E)
    x0 = rnd(T, H).bfloat16()
    ws = [torch.empty(moe.moe_grouped_ffn_w8a8_workspace(layers[0], T, k), dtype=torch.uint8, device=DEV) for _ in range(n)]

    def run():
        h = moe.moe_norm(x0, pre[0], codes=True)
        x, got = x0, []
        for l in range(n):
            lg = moe.moe_linear_int8(h.xq, h.sx, qr, sr_, dtype=torch.float32)
            ids, w = moe.moe_route_scored(lg, k, bias=bias, score=moe.MOE_SCORE_SIGMOID, n_group=4, topk_group=2,
                                          group_top=2, scale=1.5)
            counts, offsets, srt, rp = moe.moe_permute(ids, E)
            rows = moe.moe_grouped_ffn_w8a8(layers[l], h.xq, h.sx, k, counts, offsets, srt, ws=ws[l])
            h = moe.moe_combine_norm(rows, rp, w, x, post[l], next_weight=pre[l + 1], codes=True)
            x = h.y
            got += [ids, w, h.y, h.xn, h.xq, h.sx]
        return got

    return run


@pytest.mark.parametrize("T", [1, 3, 40, 130])
def test_run_together_replayed_and_on_other_streams(T):
    run = _decoder(T)
    eager = [t.clone() for t in run()]
    assert all(torch.isfinite(t.float()).all() for t in eager)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for _ in range(3):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
    # two streams at once, each with its own buffers
    other = _decoder(T)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        a = run()
    with torch.cuda.stream(s2):
        b = other()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, eager)) and all(torch.equal(p, q) for p, q in zip(b, eager))
    no_device_error()


def test_norm_codes_of_tiny_rows():
    """Rows whose scale has few bits left, or none: codes stay in range and stand for the values."""
    H = 128
    x = torch.zeros((6, H), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(DEV).manual_seed(1)
    for t, size in enumerate([1e-36, 1e-38, 1e-39, 1e-40, 0.0]):
        x[t] = (size * torch.randn(H, device=DEV, generator=g)).bfloat16()
    x[5, 3] = 1e-39
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    out = moe.moe_norm(x, w, eps=1.0, codes=True)  # r = 1: n is x
    n, q, s = f64(x), f64(out.xq), f64(out.sx)[:, None]
    assert np.abs(q).max() <= 127
    # half a code, and what 1 / 127 of a maximum of 2^-149 steps loses in sx (half a step of it a code)
    assert np.all(np.abs(q * s - n) <= 0.51 * s + 127 * 2.0 ** -150 + 2.0 ** -149)


@pytest.mark.parametrize("T", [2, 60])
def test_calls_on_a_given_stream(T):
    """`stream=`: results as on the current one, with outputs and workspace made by the
    call, while the current stream keeps allocating and writing."""
    E, H, I, k = 8, 256, 128, 2
    L, _ = int8_layer(E, H, I, seed=41)
    g = torch.Generator(DEV).manual_seed(T)
    x = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    nw = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    lg = torch.randn(T, E, device=DEV, generator=g)

    def run(stream):
        h = moe.moe_norm(x, nw, codes=True, stream=stream)
        y = moe.moe_linear_int8(h.xq, h.sx, h.xq, h.sx, stream=stream)
        ids, w = moe.moe_route_scored(lg, k, stream=stream)
        counts, offsets, srt, rp = perm if stream is not None else moe.moe_permute(ids, E)
        rows = moe.moe_grouped_ffn_w8a8(L, h.xq, h.sx, k, counts, offsets, srt, stream=stream)
        end = moe.moe_combine_norm(rows, rp, w, x, nw, next_weight=nw, codes=True, stream=stream)
        return [h.xn, h.xq, h.sx, y, ids, w, end.y, end.xn, end.xq, end.sx], (counts, offsets, srt, rp)

    want, perm = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        got, _ = run(side)
        noise = [torch.full((T, H), 3.0, device=DEV) for _ in range(8)]  # what the current stream does meanwhile
        del noise
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [1, 3, 40, 300])
def test_operands_rewritten_between_calls(T):
    """Calls in a row on one stream whose weights and codes the launch before writes."""
    N, K, n = 300, 1024, 12
    g = torch.Generator(DEV).manual_seed(T)
    ws = [torch.randn(N, K, device=DEV, generator=g).bfloat16() for _ in range(2)]
    xs = [torch.randn(T, K, device=DEV, generator=g).bfloat16() for _ in range(2)]
    nw = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    wq, sw = torch.empty((N, K), dtype=torch.int8, device=DEV), torch.empty(N, device=DEV)
    xq, sx = torch.empty((T, K), dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)

    def step(i, wait):
        moe.moe_quantize_int8(ws[i % 2], q=wq, scale=sw)
        if wait:
            torch.cuda.synchronize()
        moe.moe_norm(xs[(i // 2) % 2], nw, codes=True, want_xn=False, xq=xq, sx=sx)
        if wait:
            torch.cuda.synchronize()
        return moe.moe_linear_int8(xq, sx, wq, sw)

    want = [step(i, True).clone() for i in range(4)]
    torch.cuda.synchronize()
    got = [step(i, False) for i in range(n)]
    torch.cuda.synchronize()
    assert all(torch.equal(got[i], want[i % 4]) for i in range(n))


def test_run_together_against_the_formulas():
    """One block, each step held to its reference on the step's own inputs."""
    T, E, H, I, k = 9, 16, 256, 128, 4
    L, pieces = int8_layer(E, H, I, seed=30)
    r = np.random.default_rng(8)
    xt, xv = bf16(r.standard_normal((T, H)))
    nw, nv = bf16(1 + 0.1 * r.standard_normal(H))
    h = moe.moe_norm(xt, nw, codes=True)
    check_next(h, xv, nv, 1e-6, 0.0)
    wr = dev((0.1 * r.standard_normal((E, H))).astype(np.float32)).bfloat16()
    qr, sr_ = moe.moe_quantize_int8(wr)
    lg = moe.moe_linear_int8(h.xq, h.sx, qr, sr_, dtype=torch.float32)
    ids, w = moe.moe_route_scored(lg, k)
    rid, rw = ref.route(lg.cpu().numpy(), k)
    assert np.array_equal(ids.cpu().numpy(), rid)
    counts, offsets, srt, rp = moe.moe_permute(ids, E)
    rows = moe.moe_grouped_ffn_w8a8(L, h.xq, h.sx, k, counts, offsets, srt)
    check_ffn(L, pieces, h.xq.cpu().numpy(), h.sx.cpu().numpy(), rid, rows, rp)
    out = moe.moe_combine_norm(rows, rp, w, xt, nw, next_weight=nw, codes=True)
    z, mag = ref.combine(rows.cpu().numpy(), rp.cpu().numpy(), w.cpu().numpy())
    y, tol = ref.after_block(z, mag, xv, nv, None, None, 1e-6, 0.0, 1.0, 1.0)
    assert np.all(np.abs(f64(out.y) - y) <= ref.UBF * (np.abs(y) + tol) + tol)
    check_next(out, f64(out.y), nv, 1e-6, 0.0)
    # without its norms and residual the block's end is moe_combine, bit for bit
    plain = moe.moe_combine_norm(rows, rp, w, torch.zeros_like(xt))
    assert torch.equal(plain.y, moe.moe_combine(rows, rp, w))


# ------------------------------------------------------------------ NaN and infinities on their way

def test_norm_scale_of_a_row_with_a_nan():
    """codes of 0 alone would turn the row into zeros: its scale is NaN."""
    for T, H in ((5, 128), (300, 2816), (5, 8256), (300, 16384)):
        r = np.random.default_rng([T, H])
        xt, _ = bf16(r.standard_normal((T, H)))
        w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
        clean = moe.moe_norm(xt, w, codes=True)
        bad = torch.zeros(T, dtype=torch.bool, device=DEV)
        for t, c, v in ((1, H - 1, float("nan")), (2, 0, float("inf")), (4, H // 2, float("-inf"))):
            xt[t, c] = v
            bad[t] = True
        out = moe.moe_norm(xt, w, codes=True)
        assert torch.isnan(out.sx[bad]).all() and (out.xq[bad] == 0).all()
        assert torch.equal(out.sx[~bad], clean.sx[~bad]) and torch.equal(out.xq[~bad], clean.xq[~bad])
        # and the product of such a row is NaN
        y = moe.moe_linear_int8(out.xq, out.sx, clean.xq[:5].contiguous(), clean.sx[:5].contiguous())
        assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad].float()).all()


@pytest.mark.parametrize("T", [2, 6, 70])
@pytest.mark.parametrize("I", [128, 832])
def test_ffn_w8a8_token_without_a_number(T, I):
    E, H, k = 4, 128, 2
    L, _ = int8_layer(E, H, I, seed=12)
    xq, sx = tokens(T, H, seed=13)
    r = np.random.default_rng(T)
    ids = np.argsort(r.random((T, E)), axis=1)[:, :k].astype(np.int32)
    counts, offsets, sr, rp = moe.moe_permute(dev(ids), E)
    clean = moe.moe_grouped_ffn_w8a8(L, dev(xq), dev(sx), k, counts, offsets, sr)
    for v in (float("nan"), float("inf")):
        s2 = sx.copy()
        s2[1] = v
        rows = moe.moe_grouped_ffn_w8a8(L, dev(xq), dev(s2), k, counts, offsets, sr)
        bad = torch.zeros(T * k, dtype=torch.bool, device=DEV)
        bad[rp[k:2 * k].long()] = True
        assert torch.isnan(rows[bad]).all() and torch.equal(rows[~bad], clean[~bad])
    no_device_error()


# ------------------------------------------------------------------ codes next to a half

def exact_codes(x, w):
    """Codes of the norm of rows x (bf16 values, offset 0): n / sx = 127 x w / max |x w|, in which the row's norm
    cancels.  A product of two bf16 values has 16 bits, so fp64 holds the quotient to far more than the 2^-25 by which
    one that is no half differs from it, and a half exactly."""
    p = x * w
    return np.rint(127.0 * p / np.abs(p).max(1, keepdims=True))


@pytest.mark.parametrize("T,H", [(1, 64), (5, 2816), (300, 1024), (1023, 2816), (2, 8256), (258, 16384)])
def test_norm_codes_are_the_nearest(T, H):
    r = np.random.default_rng([T, H])
    wt, wv = bf16(1.0 + 0.3 * r.standard_normal(H))
    xt, xv = bf16(r.standard_normal((T, H)) * np.exp(r.standard_normal((T, 1))))
    out = moe.moe_norm(xt, wt, codes=True)
    assert np.array_equal(f64(out.xq), exact_codes(xv, wv))
    # ties: whole numbers under a maximum of 254, every odd one of them a half of a code
    one, ov = bf16(np.ones(H))
    v = r.integers(-253, 254, (T, H)).astype(np.float64)
    v[:, 5] = 254.0
    xt, xv = bf16(v)
    assert np.array_equal(f64(moe.moe_norm(xt, one, codes=True).xq), exact_codes(xv, ov))
    # behind a block
    z, _ = bf16(r.standard_normal((T, H)))
    res, _ = bf16(r.standard_normal((T, H)))
    out = moe.moe_residual_norm(z, res, wt, next_weight=wt, codes=True, want_xn=False)
    assert np.array_equal(f64(out.xq), exact_codes(f64(out.y), wv))
    k = 3
    rows, pos = dev(r.standard_normal((T * k, H)).astype(np.float32)), dev(r.permutation(T * k).astype(np.int32))
    out = moe.moe_combine_norm(rows, pos, dev(r.random((T, k)).astype(np.float32)), res, next_weight=wt, codes=True)
    assert np.array_equal(f64(out.xq), exact_codes(f64(out.y), wv))


@pytest.mark.parametrize("lo,hi", [(120.0, 127.9), (-120.0, -100.0), (-60.0, 60.0)])
def test_norm_codes_of_large_and_small_weights(lo, hi):
    """Weights whose products with a row leave little room below the largest fp32 number, or above the least."""
    H = 128
    r = np.random.default_rng(2)
    wt, wv = bf16(np.exp2(hi - np.minimum(8.0, hi - lo) * r.random(H)))
    xt, xv = bf16(np.where(r.random((3, H)) < 0.5, -1.0, 1.0))
    out = moe.moe_norm(xt, wt, codes=True)
    assert np.array_equal(f64(out.xq), exact_codes(xv, wv))
    # rsqrt (the 64-bit reference's own square root included) and two products, then a division
    n, rel = ref.norm(xv, wv, 1e-6, 0.0)
    assert np.all(np.abs(f64(out.sx) - np.abs(n).max(1) / 127.0) <= (rel + 2 * ref.U32) * np.abs(n).max(1) / 127.0)


@pytest.mark.parametrize("T", [1, 3, 70])
@pytest.mark.parametrize("I", [64, 832])
def test_ffn_w8a8_codes_next_to_a_half(T, I):
    """Rows of h that are whole numbers (the gate is large, so gelu is the identity) under scales that are odd whole
    numbers, every value a half of a code; the second product writes the codes out."""
    E, H, k = 2, 64, 1
    r = np.random.default_rng([T, I])
    for s in (7, 11, 23):
        # h_i = 16 u_i with max u = 254 s: sh = 32 s, h / sh = u / (2 s)
        u = s * r.integers(-253, 254, I)
        u[0] = 254 * s
        q13 = np.zeros((E, 2 * I, H), np.int8)
        q13[:, :I, 0] = 16
        left = u.copy()
        for j in range(H):
            q13[:, I:, j] = np.clip(left, -127, 127)
            left = left - np.clip(left, -127, 127)
        assert not left.any()
        q2 = np.zeros((E, H, I), np.int8)
        cols = r.permutation(I)[:H]
        cols[0] = 0
        q2[:, np.arange(H), cols] = 1
        one = lambda *sh: np.ones(sh, np.float32)  # noqa: E731
        eb = (moe.moe_expert_bytes(moe.MOE_W_INT8, H, I) + 255) // 256 * 256
        blob = np.concatenate([v.view(np.uint8).ravel() for v in (q13[0], one(2 * I), q2[0], one(H))])
        home = np.zeros((E, eb), np.uint8)
        home[:, :blob.size] = blob
        L = moe.MoeLayer(moe.MOE_W_INT8, E, H, I, dev(home.ravel()), expert_bytes=eb)
        xq = np.ones((T, H), np.int8)
        ids = dev(r.integers(0, E, (T, k)).astype(np.int32))
        counts, offsets, sr, rp = moe.moe_permute(ids, E)
        rows = moe.moe_grouped_ffn_w8a8(L, dev(xq), dev(np.ones(T, np.float32)), k, counts, offsets, sr)
        want = np.rint(u[cols] / (2.0 * s)) * (32.0 * s)  # whole numbers below 2^24: exact in fp32
        assert np.array_equal(f64(rows), np.broadcast_to(want, (T, H)))
    no_device_error()


# ------------------------------------------------------------------ sizes past the repository's own shape

@pytest.mark.parametrize("E,H,I,k", [(3, 128, 832, 2), (3, 3136, 64, 2), (2, 4096, 2048, 1), (2, 64, 16384, 1),
                                     (2, 16384, 64, 2)])
@pytest.mark.parametrize("T", [1, 7, 20, 45, 90])
def test_ffn_w8a8_long_rows(E, H, I, k, T):
    """Rows of h that no warp holds in registers, weight rows that take a second round of loads."""
    L, pieces = int8_layer(E, H, I, seed=E + H + I)
    xq, sx = tokens(T, H, seed=k)
    r = np.random.default_rng([T, H, I])
    ids = np.argsort(r.standard_normal((T, E)), axis=1)[:, :k].astype(np.int32)
    counts, offsets, sr, rp = moe.moe_permute(dev(ids), E)
    rows = moe.moe_grouped_ffn_w8a8(L, dev(xq), dev(sx), k, counts, offsets, sr)
    check_ffn(L, pieces, xq, sx, ids, rows, rp, only={0, T // 2, T - 1})
    no_device_error()


@pytest.mark.parametrize("T", [3, 4, 113, 128])
@pytest.mark.parametrize("N,K", [(1, 16), (7, 64), (33, 80), (130, 272), (300, 1040), (64, 2816), (129, 528),
                                 (1409, 2816), (5000, 1040)])
def test_linear_int8_block_sizes(T, N, K):
    """The dp4a product of four tokens, and the largest blocks of the split product."""
    test_linear_int8(T, N, K)


@pytest.mark.parametrize("T", [3, 70])
def test_linear_int8_inside_a_buffer(T):
    N, K = 37, 96
    r = np.random.default_rng(T)
    xq, wq = random_codes(r, T, K), random_codes(r, N, K)
    sx, sw = (0.5 + r.random(T)).astype(np.float32), (0.5 + r.random(N)).astype(np.float32)
    buf = torch.full(((T * N + 15) // 8 * 8 + 64,), 7.0, device=DEV)
    y = buf[32:32 + T * N].view(T, N)
    moe.moe_linear_int8(dev(xq), dev(sx), dev(wq), dev(sw), y=y)
    want = ref.linear(xq, sx, wq, sw)
    assert np.all(np.abs(f64(y) - want) <= 3 * (1 + 1e-6) * ref.U32 * np.abs(want))
    assert (buf[:32] == 7).all() and (buf[32 + T * N:] == 7).all()


# ------------------------------------------------------------------ offsets past 32 bits

def test_linear_int8_offsets_past_32_bits():
    g = torch.Generator(DEV).manual_seed(5)
    code = lambda *s: torch.randint(-127, 128, s, generator=g, dtype=torch.int8, device=DEV)  # noqa: E731
    # a weight of 4.6 GB, by each of the kernels for few tokens
    N, K = 70001, 65536
    wq, sw = code(N, K), torch.ones(N, device=DEV)
    for T in (2, 5):
        xq = code(T, K)
        y = moe.moe_linear_int8(xq, torch.ones(T, device=DEV), wq, sw, dtype=torch.float32)
        for n in (0, 32767, 32768, 65535, 65536, N - 1):  # 32768 and 65536 start at 2^31 and 2^32 bytes
            want = (xq.double() * wq[n].double()).sum(1)
            assert bool(((y[:, n].double() - want).abs() <= ref.U32 * want.abs()).all())
    del wq, y
    # an output of 2.5e9 values
    T, N, K = 50001, 50003, 64
    xq, wq = code(T, K), code(N, K)
    y = moe.moe_linear_int8(xq, torch.ones(T, device=DEV), wq, torch.ones(N, device=DEV), dtype=torch.float32)
    for t in (0, 21473, 42947, 42949, 42950, T - 1):  # (rows around 2^30, 2^31 values and the end)
        assert torch.equal(y[t].double(), wq.double() @ xq[t].double())  # sums below 2^24
    no_device_error()


def test_norm_offsets_past_32_bits():
    T, H = 140001, 16384
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    x = torch.randn((64, H), device=DEV, generator=torch.Generator(DEV).manual_seed(6)).bfloat16()
    x = x.repeat((T + 63) // 64, 1)[:T]
    out = moe.moe_norm(x, w, codes=True)
    for lo in (0, 65472, 131072, T - 64):
        part = moe.moe_norm(x[lo:lo + 64], w, codes=True)
        for a, b in ((out.xn, part.xn), (out.xq, part.xq), (out.sx, part.sx)):
            assert torch.equal(a[lo:lo + 64], b)


def test_route_scored_offsets_past_32_bits():
    T, E, k = 4200001, 1024, 1
    lg = torch.zeros((T, E), device=DEV)
    at = torch.arange(T, device=DEV)
    lg[at, at % E] = 3.0
    ids, _ = moe.moe_route_scored(lg, k)
    assert torch.equal(ids[:, 0].long(), at % E)


def test_ffn_w8a8_offsets_past_32_bits():
    """Rows of 5.4 GB; routes of one token's codes, so that every expert's rows are alike."""
    E, H, I, k = 3, 16384, 64, 1
    T = 82001
    L, pieces = int8_layer(E, H, I, seed=77)
    xq, sx = tokens(1, H, seed=1)
    ids = (torch.arange(T, device=DEV) % E).to(torch.int32)[:, None]
    counts, offsets, sr, rp = moe.moe_permute(ids, E)
    rows = moe.moe_grouped_ffn_w8a8(L, dev(xq).repeat(T, 1), dev(sx).repeat(T), k, counts, offsets, sr)
    at = offsets.tolist()
    for e in range(E):
        row, tol = ref.ffn_row(xq[0], sx[0], *(p[e] for p in pieces))
        assert np.all(np.abs(f64(rows[at[e]]) - row) <= tol)
        assert bool((rows[at[e]:at[e + 1]] == rows[at[e]]).all())
    no_device_error()
