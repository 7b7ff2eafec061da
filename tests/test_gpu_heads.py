"""Dropout, low-rank adapters and head rotation against their 64-bit definitions (MI355X)."""
import math

import numpy as np
import pytest
import torch

import heads_util as hu
import lut_sketched_matmul_amd as skm

pytestmark = pytest.mark.gpu

T = hu.T
NAN, INF = float("nan"), float("inf")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, sigma, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def seed_of(k, s=7):
    return torch.tensor([k, s], dtype=torch.int64, device="cuda")


# ---- dropout -----------------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("count", [1, 7, 8, 9, 2049, 1 << 16])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
@pytest.mark.parametrize("res", [False, True])
def test_dropout(dt, count, p, res):
    g = gen(count)
    x, r = normal(g, (count,), 3.0, T[dt]), normal(g, (count,), 1.0, T[dt])
    seed = seed_of(-(1 << 40) - 3, (1 << 50) + 11)
    y = skm.sketch_dropout(x, p, seed, residual=r if res else None)
    mul = hu.multiplier((count,), p, seed.tolist(), "cuda")
    d = x.double() * mul
    want = d + r.double() if res else d
    # the quotient's half step, the sum's, the result's rounding to its type
    bound = hu.U[T[dt]] * want.abs() * (1 + 2.0 ** -7) + hu.E * (d.abs() + want.abs()) * (res or dt != "f32") + hu.SUB[T[dt]]
    assert hu.off(y, (want, bound)) <= 0
    if not res:
        assert bool(((y == 0) == ((mul == 0) | (x == 0))).all())


def test_dropout_words_match_python_integers():
    seed = [0x1234567890ABCDEF, -5]
    h = hu.halves(8 * (1 << 33), 8, seed)  # (block numbers past 32 bits)
    M = (1 << 64) - 1
    w = hu.philox(seed[0] & M, 1 << 33, seed[1] & M)
    assert [int(v) for v in h] == [v for x in w for v in (x & 0xFFFF, x >> 16)]


def test_dropout_drops_what_is_not_finite_and_keeps_the_rest():
    x = torch.full((4096,), NAN, device="cuda")
    x[::2] = INF
    seed = seed_of(3)
    mul = hu.multiplier((4096,), 0.5, seed.tolist(), "cuda")
    for dt in T.values():
        y = skm.sketch_dropout(x.to(dt), 0.5, seed)
        assert bool((y[mul == 0] == 0).all()) and bool((~torch.isfinite(y[mul > 0])).all())


def test_dropout_seed_is_read_on_the_device():
    x = torch.ones(1 << 12, device="cuda", dtype=torch.bfloat16)
    seed = seed_of(1)
    outs = []
    for k in range(3):
        seed[1] = k
        outs.append(skm.sketch_dropout(x, 0.5, seed))
    for k, y in enumerate(outs):
        mul = hu.multiplier((1 << 12,), 0.5, [1, k], "cuda")
        assert bool((y.double() == mul).all())
    assert not bool((outs[0] == outs[1]).all())


def test_dropout_past_32_bits():
    n = (1 << 31) + 4097
    x = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    y = skm.sketch_dropout(x, 0.25, seed_of(99, 1))
    for first in (0, (1 << 31) - 4096, n - 4097 - 7):
        first -= first % 8
        c = min(4096, n - first)
        keep = torch.from_numpy(hu.halves(first, c, [99, 1]) >= 16384).to("cuda")
        assert bool(((y[first:first + c] != 0) == keep).all())


# ---- adapters -------------------------------------------------------------------------------

def case(seed, m, d, n, r, S, dt, ids="mixed", p=0.0, scale=True, base=True, back=True):
    g = gen(seed)
    t = T[dt]
    c = dict(X=normal(g, (m, d), 1.0, t), A=normal(g, (S, r, d), 1 / math.sqrt(d), t), B=normal(g, (S, n, r), 0.1, t),
             base=normal(g, (m, n), 1.0, t) if base else None, scale=None, ids=None, p=p, seed=[seed * 7 + 1, 5])
    if scale:
        c["scale"] = 0.5 + torch.rand(S, generator=g, device="cuda")
    rng = np.random.default_rng(seed)
    if ids == "mixed":
        v = rng.integers(-1, S + 1, m)  # (S is no adapter either)
    elif ids == "ragged":
        cuts = np.sort(rng.integers(0, m + 1, 4))
        v = rng.integers(-1, S, 5)[np.searchsorted(cuts, np.arange(m), side="right")]
    elif ids == "none":
        v = np.full(m, -1)
    elif ids == "last":
        v = np.full(m, S - 1)
    else:
        v = None
    if v is not None:
        c["ids"] = torch.from_numpy(v.astype(np.int32)).to("cuda")
    if back:
        c["dY"] = normal(g, (m, n), 0.1, t)
        c["base_dx"] = normal(g, (m, d), 0.1, torch.float32) if base else None
    return c


def forward(c, **kw):
    return skm.sketch_adapter_fwd(c["X"], c["A"], c["B"], c["base"], adapter=c["ids"], scale=c["scale"], p=c["p"],
                                  seed=torch.tensor(c["seed"], device="cuda") if c["p"] else None, **kw)


def backward(c, H, **kw):
    return skm.sketch_adapter_bwd(c["dY"], c["X"], H, c["A"], c["B"], c["base_dx"], adapter=c["ids"], scale=c["scale"],
                                  p=c["p"], seed=torch.tensor(c["seed"], device="cuda") if c["p"] else None, **kw)


def check(c):
    Y, H = forward(c, need_h=True)
    want = hu.adapter64(c)
    got = dict(Y=Y, H=H)
    if "dY" in c:
        # (the backward's own rounding: from the H it was given, whose bound is in dB's)
        got["dX"], got["dA"], got["dB"] = backward(c, H)
    for k, v in got.items():
        assert hu.off(v, want[k]) <= 0, (k, hu.off(v, want[k]))
    return got


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("m,d,n,r,S,ids", [
    (1, 32, 1, 1, 1, None), (1, 64, 8, 16, 1, "last"), (2, 96, 17, 3, 2, "mixed"), (15, 128, 130, 8, 4, "mixed"),
    (16, 256, 127, 16, 3, "ragged"), (17, 1024, 129, 12, 40, "mixed"), (33, 544, 256, 24, 5, "mixed"),
    (64, 4096, 1000, 16, 64, "mixed"), (100, 288, 4097, 33, 7, "ragged"), (130, 320, 72, 64, 2, "mixed"),
    (50, 64, 300, 65, 3, "mixed"), (40, 160, 264, 128, 2, "ragged"), (300, 512, 640, 16, 1, None),
    (70, 96, 40, 4, 300, "mixed"), (9, 64, 64, 5, 2, "none"), (257, 2080, 513, 20, 3, "last")])
def test_adapter(dt, m, d, n, r, S, ids):
    check(case(m + r, m, d, n, r, S, dt, ids))


@pytest.mark.parametrize("dt,n,r,ids,p", [("bf16", 320, 16, None, 0.0), ("f16", 321, 12, "ragged", 0.1),
                                          ("bf16", 201, 40, "mixed", 0.25), ("f16", 128, 64, None, 0.5),
                                          ("bf16", 136, 100, "ragged", 0.05)])
def test_adapter_many_tokens(dt, n, r, ids, p):
    """Two tiles a wave, several chunks and partial gradients."""
    check(case(r, 5003, 352, n, r, 3, dt, ids, p=p))


@pytest.mark.parametrize("dt,m,d,n,r,S,ids,p", [("bf16", 700, 2080, 520, 64, 70, "mixed", 0.0),
                                                ("f16", 530, 4096, 264, 33, 5, "ragged", 0.1),
                                                ("bf16", 513, 4096, 1001, 16, 600, "mixed", 0.0),
                                                ("f16", 512, 1056, 300, 48, 9, "ragged", 0.0),
                                                ("bf16", 10007, 64, 2056, 16, 2, "ragged", 0.0),
                                                ("f16", 33001, 32, 200, 24, 1, None, 0.0)])
def test_adapter_ranges_and_many_adapters(dt, m, d, n, r, S, ids, p):
    """The contraction in several ranges, added up in between; a tile with an adapter per token."""
    check(case(d, m, d, n, r, S, dt, ids, p=p))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("p", [0.1, 0.5, 1.0])
def test_adapter_dropout(dt, p):
    c = case(11, 37, 224, 60, 10, 2, dt, "mixed", p=p)
    got = check(c)
    # the mask is sketch_dropout's
    ones = torch.ones_like(c["X"])
    kept = skm.sketch_dropout(ones, p, torch.tensor(c["seed"], device="cuda")) != 0
    c2 = dict(c, X=torch.where(kept, c["X"], NAN))
    assert torch.equal(forward(c2)[0], got["Y"])


@pytest.mark.parametrize("what", ["base", "scale", "ids"])
def test_adapter_left_out_arguments(what):
    c = case(5, 40, 128, 96, 16, 2, "bf16", None if what == "ids" else "mixed", scale=what != "scale", base=what != "base")
    check(c)


def test_adapter_scales_of_f16():
    """h far outside f16's range: every token is scaled by itself."""
    c = case(3, 48, 256, 200, 16, 3, "f16", "mixed")
    k = torch.arange(48, device="cuda")
    c["X"] = (c["X"].float() * torch.exp2((k % 12 - 6).float() * 2)[:, None]).half()
    c["A"] *= 64
    c["B"] = (c["B"].float() * 2.0 ** -6).half()
    c["scale"][1] = 2.0 ** 20
    c["scale"][2] = 2.0 ** -30
    check(c)


def test_adapter_rows_do_not_mix():
    """What one token or adapter holds reaches only its own rows."""
    c = case(8, 64, 256, 264, 16, 4, "bf16", "mixed", base=False)
    clean = dict(zip(("Y", "H", "dX", "dA", "dB"), (*forward(c, need_h=True), None, None, None)))
    clean["dX"], clean["dA"], clean["dB"] = backward(c, clean["H"])
    ids = c["ids"]
    bad = int(torch.nonzero(ids == 2)[0])
    none = int(torch.nonzero((ids < 0) | (ids >= 4))[0])
    X, dY, A = c["X"].clone(), c["dY"].clone(), c["A"].clone()
    X[bad], X[none], dY[none] = INF, NAN, NAN
    A[3, 5] = NAN
    c2 = dict(c, X=X, A=A, dY=dY)
    Y, H = forward(c2, need_h=True)
    dX, dA, dB = backward(c2, H)
    # (token `none` has no base here: its output is zero, its gradient too)
    same = (ids != 3) & (torch.arange(64, device="cuda") != bad)
    assert torch.equal(Y[same], clean["Y"][same]) and torch.equal(dX[ids < 3], clean["dX"][ids < 3])
    assert not bool(torch.isfinite(Y[bad]).any()) and not bool(torch.isfinite(Y[ids == 3]).any())
    for s in (0, 1):
        assert torch.equal(dA[s], clean["dA"][s]) and torch.equal(dB[s], clean["dB"][s])
    assert bool((Y[none] == 0).all()) and bool((H[none] == 0).all())


def test_adapter_without_tokens_has_zero_gradients():
    c = case(4, 30, 96, 50, 8, 6, "f16", "last")
    _, H = forward(c, need_h=True)
    _, dA, dB = backward(c, H)
    assert bool((dA[:5] == 0).all()) and bool((dB[:5] == 0).all()) and bool((dA[5] != 0).any())


@pytest.mark.parametrize("ids,m", [(None, 100), ("mixed", 100), ("ragged", 3000), (None, 3000)])
def test_adapter_accumulates_and_repeats(ids, m):
    c = case(m, m, 160, 72, 16, 3, "bf16", ids)
    _, H = forward(c, need_h=True)
    _, dA, dB = backward(c, H)
    _, dA2, dB2 = backward(c, H)
    assert torch.equal(dA, dA2) and torch.equal(dB, dB2)
    a0, b0 = torch.randn_like(dA), torch.randn_like(dB)
    _, a, b = backward(c, H, da_out=a0.clone(), db_out=b0.clone(), accumulate=True, need_dx=False)
    for got, first, more in ((a, a0, dA), (b, b0, dB)):
        # added in fp32, in one addition or as the first of the chunks' sums
        assert float((got - (first + more)).abs().max()) <= 64 * 2.0 ** -24 * float(first.abs().max() + more.abs().max())


def test_adapter_parts_alone():
    c = case(6, 90, 128, 104, 16, 2, "f16", "ragged", p=0.1)
    _, H = forward(c, need_h=True)
    full, want = backward(c, H), hu.adapter64(c)
    for need in ((True, False, False), (False, True, False), (False, False, True)):
        got = backward(c, H if need[2] else None, need_dx=need[0], need_da=need[1], need_db=need[2])
        for g, k, on in zip(got, ("dX", "dA", "dB"), need):  # (sums may be cut into other chunks)
            assert (g is None) if not on else hu.off(g, want[k]) <= 0
        assert not need[0] or torch.equal(got[0], full[0])


def test_adapter_in_place_and_empty():
    c = case(9, 50, 96, 75, 8, 2, "bf16", "mixed", back=False)
    Y, _ = forward(c)
    own = dict(c, base=c["base"].clone())
    got, _ = forward(own, out=own["base"])
    assert got is own["base"] and torch.equal(got, Y)
    e = torch.empty
    z = dict(dtype=torch.bfloat16, device="cuda")
    Y, H = skm.sketch_adapter_fwd(e((0, 96), **z), c["A"], c["B"], e((0, 75), **z), need_h=True)
    dX, dA, dB = skm.sketch_adapter_bwd(e((0, 75), **z), e((0, 96), **z), H, c["A"], c["B"])
    assert Y.shape == (0, 75) and H.shape == (0, 8) and dX.shape == (0, 96)
    assert bool((dA == 0).all()) and bool((dB == 0).all())


def test_adapter_gradients_against_differences():
    """<dY, Y(v + e u) - Y(v - e u)> / 2 e of the definition in 64 bits against <gradient, u>: the definition is
    linear in each of X, A and B, so the difference is exact up to the inputs' own rounding (none in 64 bits)."""
    c = case(2, 12, 64, 24, 8, 2, "bf16", "mixed", p=0.25, base=False)
    _, H = forward(c, need_h=True)
    grads = dict(zip("XAB", backward(c, H)))
    g = gen(1)
    for k, gr in grads.items():
        u = torch.randn(c[k].shape, generator=g, device="cuda").double()
        ys = []
        for e in (1.0, -1.0):
            c2 = {q: v.double() if q in "XAB" else v for q, v in c.items() if q not in ("dY",)}
            c2[k] = c2[k] + e * u
            c2["X"], c2["dY"] = c2["X"], None
            hu.U[torch.float64], hu.SUB[torch.float64] = 0.0, 0.0
            ys.append(hu.adapter64(c2)["Y"][0])
        want = float(((ys[0] - ys[1]) / 2 * c["dY"].double()).sum())
        terms = gr.double() * u
        # dX is rounded to bf16, the others to fp32 after sums of up to 64 terms
        rel = 2.0 ** -8 if k == "X" else 2.0 ** -16
        assert abs(float(terms.sum()) - want) <= rel * float(terms.abs().sum())


def test_adapter_past_32_bits():
    """Rows of base, Y and dY behind 2^31 elements."""
    m, n, d, r = 70000, 32000, 64, 8
    t = torch.bfloat16
    g = gen(1)
    X, A, B = normal(g, (m, d), 1.0, t), normal(g, (1, r, d), 0.1, t), normal(g, (1, n, r), 0.1, t)
    Y, H = skm.sketch_adapter_fwd(X, A, B, need_h=True)
    rows = torch.tensor([0, 5, 67107, 67109, 69999], device="cuda")
    sub = dict(X=X[rows], A=A, B=B, base=None, ids=None, scale=None, p=0.0, seed=[0, 0])
    want = hu.adapter64(sub)
    assert hu.off(Y[rows], want["Y"]) <= 0 and hu.off(H[rows], want["H"]) <= 0
    # one token's gradient among zeros: dB is that token's alone
    Y.zero_()
    Y[69999] = 1.0
    dX, dA, dB = skm.sketch_adapter_bwd(Y, X, H, A, B)
    h = H[69999].double()
    assert hu.off(dB[0], (h.expand(n, r), 2.0 ** -23 * h.abs().expand(n, r))) <= 0
    assert bool((dX[:69999] == 0).all()) and bool((dX[69999] != 0).any())


# ---- rotary ----------------------------------------------------------------------------------

def heads(seed, m, hq, hk, dh, dt, joined=True):
    g = gen(seed)
    if not joined:
        return normal(g, (m, hq, dh), 2.0, T[dt]), normal(g, (m, hk, dh), 2.0, T[dt]) if hk else None
    x = normal(g, (m, (hq + 2 * hk) * dh), 2.0, T[dt])
    return x[:, :hq * dh].unflatten(1, (hq, dh)), x[:, hq * dh:(hq + hk) * dh].unflatten(1, (hk, dh)) if hk else None


def freqs(rot, theta=10000.0):
    return theta ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)


def rotary_check(seed, m, hq, hk, dh, rot, dt, eps, pairs, weights=True, joined=True, far=5000):
    g = gen(seed + 1)
    q, k = heads(seed, m, hq, hk, dh, dt, joined)
    pos = torch.randint(-far, far + 1, (m,), generator=g, device="cuda")
    f = freqs(rot)
    qw = kw = None
    if eps is not None and weights:
        qw, kw = (1 + 0.3 * torch.randn(dh, generator=g, device="cuda") for _ in range(2))
    dq, dk = normal(g, (m, hq, dh), 0.1, T[dt]), normal(g, (m, hk, dh), 0.1, T[dt]) if hk else None
    yq, yk = skm.sketch_rotary_fwd(q, k, pos, f, qw, kw, eps=eps, pairs=pairs)
    gq, gk, gqw, gkw = skm.sketch_rotary_bwd(dq, dk, q, k, pos, f, qw, kw, eps=eps, pairs=pairs)
    for x, w, dy, y, dx, dw in ((q, qw, dq, yq, gq, gqw), (k, kw, dk, yk, gk, gkw)):
        if x is None:
            assert y is None and dx is None and dw is None
            continue
        want = hu.rotary64(x, w, pos, f, eps, pairs, dy)
        assert hu.off(y, want["y"]) <= 0, hu.off(y, want["y"])
        assert hu.off(dx, want["dx"]) <= 0, hu.off(dx, want["dx"])
        if eps is not None:
            assert hu.off(dw, want["dw"]) <= 0, hu.off(dw, want["dw"])
        else:
            assert dw is None


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("eps", [None, 1e-6])
@pytest.mark.parametrize("m,hq,hk,dh,rot", [(1, 1, 0, 2, 2), (1, 32, 8, 128, 128), (3, 4, 4, 64, 32), (17, 5, 1, 80, 36),
                                            (130, 6, 2, 96, 96), (33, 3, 3, 126, 126), (9, 2, 1, 256, 128),
                                            (5, 1, 1, 16, 16), (4, 2, 1, 34, 10)])
def test_rotary(dt, pairs, eps, m, hq, hk, dh, rot):
    rotary_check(m + dh, m, hq, hk, dh, rot, dt, eps, pairs)


@pytest.mark.parametrize("dh,rot", [(512, 512), (1024, 1024), (1022, 600), (300, 300), (32, 32), (510, 4)])
def test_rotary_wide_heads(dh, rot):
    rotary_check(dh, 7, 3, 2, dh, rot, "bf16", 1e-6, "halves")
    rotary_check(dh, 7, 3, 0, dh, rot, "f32", 1e-6, "neighbours")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("dh,rot", [(528, 16), (1008, 32), (514, 2), (1022, 32), (80, 20), (96, 24)])
def test_rotary_lanes_behind_a_wide_head(dh, rot, pairs, dt):
    """Heads that leave lanes of their group idle, with so many tokens that a block holds the angles of several."""
    rotary_check(dh + rot, 8200, 1, 1, dh, rot, dt, 1e-6, pairs)


def test_rotary_many_tokens_and_no_weights():
    rotary_check(1, 4099, 8, 2, 128, 128, "bf16", 1e-5, "halves", weights=False, joined=False)
    rotary_check(2, 2500, 40, 10, 64, 64, "f16", 1e-5, "neighbours")


def test_rotary_far_positions():
    """Angles of positions up to 2^40 against whole turns taken away with Python's integers and fractions."""
    from fractions import Fraction
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286, 10 ** 75)
    pos = torch.tensor([0, 1, -1, 131072, (1 << 31) + 5, -(1 << 35) - 1, 1 << 40], device="cuda")
    f = freqs(64)
    x = torch.zeros((7, 1, 64), device="cuda")
    x[..., :32] = 1.0
    y, _ = skm.sketch_rotary_fwd(x, None, pos, f)
    for t, p in enumerate(pos.tolist()):
        for i in range(0, 32, 5):
            a = Fraction(float(p) * float(f[i]))  # the fp64 product
            a = float(a - 2 * pi * round(a / (2 * pi)))
            assert abs(float(y[t, 0, i]) - math.cos(a)) <= 2.0 ** -22 and abs(float(y[t, 0, 32 + i]) - math.sin(a)) <= 2.0 ** -22


def test_rotary_in_place_and_joined_gradient():
    m, hq, hk, dh = 65, 8, 2, 128
    q, k = heads(3, m, hq, hk, dh, "bf16")
    pos, f = torch.arange(m, device="cuda"), freqs(dh)
    w = torch.ones(dh, device="cuda")
    want = skm.sketch_rotary_fwd(q, k, pos, f, w, w, eps=1e-6)
    dq, dk = torch.randn_like(want[0]), torch.randn_like(want[1])
    gq, gk, _, _ = skm.sketch_rotary_bwd(dq, dk, q, k, pos, f, w, w, eps=1e-6)
    joint = torch.full((m, (hq + 2 * hk) * dh), 7.0, device="cuda", dtype=torch.bfloat16)
    skm.sketch_rotary_bwd(dq, dk, q, k, pos, f, w, w, eps=1e-6, q_out=joint[:, :hq * dh].unflatten(1, (hq, dh)),
                          k_out=joint[:, hq * dh:(hq + hk) * dh].unflatten(1, (hk, dh)))
    assert torch.equal(joint[:, :hq * dh], gq.flatten(1)) and torch.equal(joint[:, hq * dh:(hq + hk) * dh], gk.flatten(1))
    assert bool((joint[:, (hq + hk) * dh:] == 7.0).all())
    got = skm.sketch_rotary_fwd(q, k, pos, f, w, w, eps=1e-6, q_out=q, k_out=k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0] is q


def test_rotary_leaves_other_columns_and_bad_heads_alone():
    m, h, dh = 40, 4, 64
    q, _ = heads(5, m, h, 0, dh, "f16", joined=False)
    pos, f = torch.arange(m, device="cuda"), freqs(dh)
    clean, _ = skm.sketch_rotary_fwd(q, None, pos, f, eps=1e-6)
    q2 = q.clone()
    q2[7, 2, 5] = NAN
    got, _ = skm.sketch_rotary_fwd(q2, None, pos, f, eps=1e-6)
    bad = torch.zeros((m, h), dtype=torch.bool, device="cuda")
    bad[7, 2] = True
    assert torch.equal(got[~bad], clean[~bad]) and bool(torch.isnan(got[7, 2]).all())
    # rows that start at any element
    big = torch.full((m, h * dh + 3), 9.0, device="cuda", dtype=torch.float16)
    odd = big[:, 1:1 + h * dh].unflatten(1, (h, dh))
    skm.sketch_rotary_fwd(q, None, pos, f, eps=1e-6, q_out=odd)
    assert float((odd.float() - clean.float()).abs().max()) <= 2.0 ** -10 * float(clean.float().abs().max())
    assert bool((big[:, 0] == 9).all()) and bool((big[:, 1 + h * dh:] == 9).all())


def test_rotary_accumulates_and_repeats():
    m, hq, hk, dh = 700, 6, 3, 96
    q, k = heads(4, m, hq, hk, dh, "bf16")
    pos, f = torch.arange(m, device="cuda"), freqs(dh)
    w = torch.ones(dh, device="cuda")
    dq, dk = (torch.randn((m, h, dh), device="cuda").bfloat16() for h in (hq, hk))
    a = skm.sketch_rotary_bwd(dq, dk, q, k, pos, f, w, w, eps=1e-6)
    b = skm.sketch_rotary_bwd(dq, dk, q, k, pos, f, w, w, eps=1e-6)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    s = torch.randn(dh, device="cuda")
    c = skm.sketch_rotary_bwd(dq, dk, q, k, pos, f, w, w, eps=1e-6, qw_out=s.clone(), kw_out=s.clone(), accumulate=True)
    assert torch.equal(c[2], s + a[2]) and torch.equal(c[3], s + a[3])


def test_rotary_past_32_bits():
    m, ld, dh = 70000, 32000, 128
    x = torch.zeros((m, ld), device="cuda", dtype=torch.bfloat16)
    g = gen(2)
    x[-1] = normal(g, (ld,), 1.0, torch.bfloat16)
    q = x[:, -256:].unflatten(1, (2, dh))
    pos, f = torch.arange(m, device="cuda"), freqs(dh)
    y, _ = skm.sketch_rotary_fwd(q, None, pos, f)
    want = hu.rotary64(q[-1:].contiguous(), None, pos[-1:], f, None, "halves")
    assert hu.off(y[-1:], want["y"]) <= 0 and bool((y[:-1] == 0).all())


# ---- streams, graphs, shared workspaces ------------------------------------------------------------

def test_calls_on_another_stream():
    c = case(21, 200, 256, 136, 16, 3, "bf16", "ragged", p=0.1)
    seed = torch.tensor(c["seed"], device="cuda")
    Y, H = forward(c, need_h=True)
    want = (Y, H, *backward(c, H))
    q, _ = heads(1, 200, 4, 0, 64, "bf16", joined=False)
    pos, f = torch.arange(200, device="cuda"), freqs(64)
    turned = skm.sketch_rotary_fwd(q, None, pos, f, eps=1e-6)[0]
    drop = skm.sketch_dropout(c["X"], 0.3, seed)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    args = (c["A"], c["B"], c["base"])
    Y, H = skm.sketch_adapter_fwd(c["X"], *args, adapter=c["ids"], scale=c["scale"], p=0.1, seed=seed, need_h=True, stream=s)
    got = (Y, H, *skm.sketch_adapter_bwd(c["dY"], c["X"], H, c["A"], c["B"], c["base_dx"], adapter=c["ids"],
                                         scale=c["scale"], p=0.1, seed=seed, stream=s))
    t2 = skm.sketch_rotary_fwd(q, None, pos, f, eps=1e-6, stream=s)[0]
    d2 = skm.sketch_dropout(c["X"], 0.3, seed, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(turned, t2) and torch.equal(drop, d2)


def test_captured_step_with_one_workspace():
    """Two graphs of a training step that share their workspace, replayed in turn with new inputs, ids and seeds."""
    m, d, n, r, S = 300, 256, 192, 16, 3
    cs = [case(31 + i, m, d, n, r, S, "bf16", "ragged", p=0.1) for i in range(2)]
    need = max(skm.sketch_adapter_fwd_workspace(m, n, d, r, S), skm.sketch_adapter_bwd_workspace(m, n, d, r, S))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    seeds = [torch.tensor(c["seed"], device="cuda") for c in cs]

    def step(c, seed):
        x = skm.sketch_dropout(c["X"], 0.2, seed)
        Y, H = skm.sketch_adapter_fwd(x, c["A"], c["B"], c["base"], adapter=c["ids"], scale=c["scale"], p=0.1, seed=seed,
                                      need_h=True, workspace=ws)
        y, _ = skm.sketch_rotary_fwd(Y.unflatten(1, (3, 64)), None, c["pos"], c["f"], eps=1e-6)
        gy, _, gw, _ = skm.sketch_rotary_bwd(c["dY"].unflatten(1, (3, 64)), None, Y.unflatten(1, (3, 64)), None, c["pos"],
                                             c["f"], eps=1e-6)
        return (y, gw, *skm.sketch_adapter_bwd(gy.flatten(1), x, H, c["A"], c["B"], c["base_dx"], adapter=c["ids"],
                                               scale=c["scale"], p=0.1, seed=seed, workspace=ws))

    graphs, outs = [], []
    for c, seed in zip(cs, seeds):
        c["pos"], c["f"] = torch.arange(m, device="cuda"), freqs(64)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step(c, seed)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(c, seed))
        graphs.append(g)
    for k in range(4):
        for i in (0, 1):
            seeds[i][1] += 1
            cs[i]["X"].copy_(torch.randn_like(cs[i]["X"]))
            cs[i]["ids"].copy_(torch.roll(cs[i]["ids"], 13 * k + 1))
            graphs[i].replay()
            got = [t.clone() for t in outs[i]]
            torch.cuda.synchronize()
            want = step(cs[i], seeds[i])
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (k, i)


# ---- the modules: a run of all of them as a fine-tuned attention layer uses them ------------------------

def layer_parts(dt, S=2, p=0.1):
    from lut_sketched_matmul_amd import finetune as ft, synthetic as syn
    from gpu_util import to_dev
    d, hq, hk, dh = 256, 4, 2, 64

    def sketch(name, n):
        return (to_dev(syn.random_packed_indices(name + "/i", n, d, 4), "u8"),
                to_dev(syn.random_lut(name + "/l", n, 2, 4, 0.05, "f16"), "f16").to(T[dt]))

    parts = [sketch(f"heads/{i}", n) for i, n in enumerate((hq * dh, hk * dh, hk * dh))]
    n = (hq + 2 * hk) * dh
    a = ft.SketchAdapter(n, d, 8, S, dropout=p, compute_dtype=T[dt], seed=3)
    with torch.no_grad():
        a.B_master.copy_(0.05 * torch.randn(a.B_master.shape, generator=gen(9), device="cuda"))
    a.refresh_copies()
    qkv = ft.GroupedSketchedLinear([i for i, _ in parts], [l for _, l in parts], d, 4, 2, compute_dtype=T[dt], adapter=a)
    out = ft.SketchedLinear(*sketch("heads/o", d), d, 4, 2, compute_dtype=T[dt])
    rot = ft.SketchRotary(dh, norm=True)
    drop = ft.SketchDropout(0.2, seed=4)
    return ft, qkv, a, rot, out, drop, (hq, hk, dh)


def run_layer(parts, X, ids, pos):
    ft, qkv, a, rot, out, drop, (hq, hk, dh) = parts
    q, k, v = qkv(X, ids)
    q, k = rot(q.unflatten(1, (hq, dh)), k.unflatten(1, (hk, dh)), pos)
    m = X.shape[0]
    kk, vv = (t.float().reshape(m, hk, dh).repeat_interleave(hq // hk, 1) for t in (k, v))
    s = torch.softmax((q.float().transpose(0, 1) @ kk.transpose(0, 1).transpose(1, 2).contiguous()) / dh ** 0.5, -1)
    y = (s @ vv.transpose(0, 1)).transpose(0, 1).reshape(m, hq * dh).to(X.dtype)
    return drop(out(y), X)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention_layer_of_the_modules(dt):
    """Joined q/k/v with adapters -> norm and rotation -> (plain) attention -> output projection -> dropout + residual:
    forward and gradients against the same layer in float64, and a step of the optimizer."""
    parts = layer_parts(dt)
    ft, qkv, a, rot, out, drop, (hq, hk, dh) = parts
    m, d = 70, 256
    X = normal(gen(1), (m, d), 1.0, T[dt]).requires_grad_()
    ids = torch.tensor(([0] * 30 + [1] * 25 + [-1] * 15), dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(30), torch.arange(40)]).to("cuda")
    Y = run_layer(parts, X, ids, pos)
    dY = normal(gen(2), (m, d), 0.1, T[dt])
    Y.backward(dY)

    from lut_sketched_matmul_amd import sketch_dequant
    x = X.detach().double().requires_grad_()
    W = sketch_dequant(qkv.inner.idx_packed, qkv.inner.lut, d, 4, 2).double()
    Wo = sketch_dequant(out.idx_packed, out.lut, d, 4, 2).double()
    A, B = (t.double().requires_grad_() for t in (a.A, a.B))
    mul = hu.multiplier((m, d), 0.1, [3, 0], "cuda")
    z = x @ W.T
    ad = [((x * mul) @ A[s].T) @ B[s].T for s in range(2)]
    z = z + torch.where(ids[:, None] == 0, ad[0], 0.0) + torch.where(ids[:, None] == 1, ad[1], 0.0)
    angle = pos.double()[:, None] * rot.inv_freq

    def head(u, h):
        u = u.unflatten(1, (h, dh))
        u = u / torch.sqrt((u * u).mean(2, keepdim=True) + 1e-6)
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        e, f = u[..., :dh // 2], u[..., dh // 2:]
        return torch.cat([e * c - f * s, e * s + f * c], 2)

    q, k = head(z[:, :hq * dh], hq), head(z[:, hq * dh:(hq + hk) * dh], hk).repeat_interleave(hq // hk, 1)
    v = z[:, (hq + hk) * dh:].unflatten(1, (hk, dh)).repeat_interleave(hq // hk, 1)
    s = torch.softmax(torch.einsum("thd,uhd->htu", q, k) / dh ** 0.5, -1)
    y = torch.einsum("htu,uhd->thd", s, v).reshape(m, hq * dh) @ Wo.T
    want = x + y * hu.multiplier((m, d), 0.2, [4, 0], "cuda")
    want.backward(dY.double())
    # Norms of the whole: about ten roundings of half a step one after the other (projection, rotation, attention's
    # output, output projection, sum), independent from value to value: sqrt(10) half steps and as much again
    rel = 8 * hu.U[T[dt]]
    for got, ref in ((Y, want), (X.grad, x.grad), (a.A_master.grad, A.grad), (a.B_master.grad, B.grad)):
        assert float((got.detach().double() - ref.detach()).norm()) <= rel * float(ref.detach().norm())
    opt = ft.LutAdam([a.A_master, a.B_master, rot.q_weight, rot.k_weight], lr=1e-3)
    before = a.B.clone()
    opt.step()
    assert torch.equal(a.A, a.A_master.detach().to(T[dt])) and torch.equal(a.B, a.B_master.detach().to(T[dt]))
    assert not torch.equal(before, a.B)


def test_captured_layer_draws_new_masks():
    """A captured forward of the layer: every replay has the masks of its own turn."""
    parts = layer_parts("bf16")
    m, d = 48, 256
    X = normal(gen(5), (m, d), 1.0, torch.bfloat16)
    ids, pos = torch.zeros(m, dtype=torch.int32, device="cuda"), torch.arange(m, device="cuda")
    a, drop = parts[2], parts[5]
    with torch.no_grad():
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run_layer(parts, X, ids, pos)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            Y = run_layer(parts, X, ids, pos)
        seen = []
        for k in range(4):
            at = [a.seed.state.clone(), drop.seed.state.clone()]
            g.replay()
            got = Y.clone()
            torch.cuda.synchronize()
            assert int(a.seed.state[1]) == int(at[0][1]) + 1 and int(drop.seed.state[1]) == int(at[1][1]) + 1
            a.seed.state.copy_(at[0])
            drop.seed.state.copy_(at[1])
            assert torch.equal(got, run_layer(parts, X, ids, pos))
            assert not any(torch.equal(got, o) for o in seen)
            seen.append(got)


@pytest.mark.parametrize("captured", [False, True])
def test_recomputed_layer_has_its_own_masks(captured):
    """A layer whose activations are recomputed in the backward pass (there, by autograd's own thread) gives the output
    and gradients of one that keeps them; without its masks the recomputation is refused."""
    from torch.utils.checkpoint import checkpoint
    from lut_sketched_matmul_amd import finetune
    m, d = 70, 256
    ids = torch.tensor(([0] * 30 + [1] * 25 + [-1] * 15), dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(30), torch.arange(40)]).to("cuda")
    dY = normal(gen(2), (m, d), 0.1, torch.bfloat16)

    def both(around):
        torch.manual_seed(11)
        parts = layer_parts("bf16")
        a, rot = parts[2], parts[3]
        X = normal(gen(1), (m, d), 1.0, torch.bfloat16).requires_grad_()
        leaves = [X, a.A_master, a.B_master, rot.q_weight, rot.k_weight]

        def step():  # (two runs through one layer: masks 0 and 1 of its dropouts)
            Y = around(lambda x: run_layer(parts, x, ids, pos), around(lambda x: run_layer(parts, x, ids, pos), X))
            return [Y.detach(), *torch.autograd.grad(Y, leaves, dY)]

        if not captured:
            return [step()]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        turns = []
        for _ in range(3):
            g.replay()
            turns.append([t.clone() for t in out])
            torch.cuda.synchronize()
        return turns

    def replayed(fn, X):
        return checkpoint(fn, X, use_reentrant=False, preserve_rng_state=False, context_fn=finetune.replay_masks)

    want, got = both(lambda fn, X: fn(X)), both(replayed)
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    if captured:
        assert not torch.equal(want[0][0], want[1][0])
    else:
        with pytest.raises(RuntimeError, match="recomputed"):
            both(lambda fn, X: checkpoint(fn, X, use_reentrant=False))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_in_front_of_an_adapted_layer(dt, kind):
    """norm -> projection + adapters, against the same in float64.

    Norms of the whole. The normed input is rounded (in every gradient of a weight), its gradient once more before the
    norm's backward, and each result: at most three half steps in a row. The norm's backward scales a row's error as
    the row, its weights (1 +- 0.6) those of a column by up to 1.6 / 1: twice that, and a rest for fp32 sums.
    """
    from gpu_util import to_dev
    from lut_sketched_matmul_amd import finetune as ft, sketch_dequant, synthetic as syn
    m, n, d, r, S, eps = 90, 384, 256, 8, 2, 1e-5
    idx = to_dev(syn.random_packed_indices("normed/i", n, d, 4), "u8")
    lut = to_dev(syn.random_lut("normed/l", n, 2, 4, 0.05, "f16"), "f16").to(T[dt])
    g = gen(1)
    a = ft.SketchAdapter(n, d, r, S, dropout=0.1, compute_dtype=T[dt], seed=3)
    with torch.no_grad():
        a.A_master.copy_(torch.randn(a.A_master.shape, generator=g, device="cuda") / 16)
        a.B_master.copy_(torch.randn(a.B_master.shape, generator=g, device="cuda") / 16)
    a.refresh_copies()
    norm = ft.SketchNorm(d, kind=kind, eps=eps)
    with torch.no_grad():
        norm.weight += 0.6 * (2 * torch.rand(d, generator=g, device="cuda") - 1)
    layer = ft.SketchedLinear(idx, lut, d, 4, 2, compute_dtype=T[dt], norm=norm, adapter=a)
    X = normal(g, (m, d), 2.0, T[dt]).requires_grad_()
    ids = torch.arange(m, device="cuda", dtype=torch.int32) % 3  # (2 is no adapter)
    dY = normal(g, (m, n), 0.1, T[dt])
    Y = layer(X, ids)
    Y.backward(dY)

    x, w, A, B = (t.detach().double().requires_grad_() for t in (X, norm.weight, a.A, a.B))
    W = sketch_dequant(layer.idx_packed, layer.lut, d, 4, 2).double().requires_grad_()
    c = x - x.mean(1, keepdim=True) if kind == "layer" else x
    xn = c / torch.sqrt((c * c).mean(1, keepdim=True) + eps) * w
    z = xn * hu.multiplier((m, d), 0.1, [3, 0], "cuda")
    on = [(ids == s).double()[:, None] for s in range(S)]
    want = xn @ W.T + sum(on[s] * ((z @ A[s].T) @ B[s].T) for s in range(S))
    want.backward(dY.double())
    code = sketch_codes(layer.idx_packed)
    dL = torch.zeros(n, 2, 16, device="cuda", dtype=torch.float64).scatter_add_(2, code.reshape(n, 2, d // 2),
                                                                            W.grad.reshape(n, 2, d // 2))
    pairs = [(Y, want), (X.grad, x.grad), (norm.weight.grad, w.grad), (a.A_master.grad, A.grad),
             (a.B_master.grad, B.grad), (layer.lut_master.grad, dL)]
    for got, ref in pairs:
        assert float((got.detach().double() - ref.detach()).norm()) <= 8 * hu.U[T[dt]] * float(ref.detach().norm())


def sketch_codes(idx):
    """The 4-bit indices [n, d] of packed rows."""
    return torch.stack([idx & 15, idx >> 4], 2).reshape(idx.shape[0], -1).long()
