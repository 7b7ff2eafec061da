"""accumulate=True without an output to add to: a new output starts from zeros, not from what its memory held."""
import pytest

pytestmark = pytest.mark.gpu


def test_accumulate_into_new_outputs():
    import torch as t

    import lut_sketched_matmul_amd as k
    m, n, d, b, gpr = 40, 96, 128, 4, 2
    g = t.Generator(device="cuda").manual_seed(1)
    idx = t.randint(0, 256, (n, d // 2), generator=g, device="cuda", dtype=t.uint8)
    lut = t.randn((n, gpr, 16), generator=g, device="cuda").half()
    X, dY = t.randn((m, d), generator=g, device="cuda").half(), t.randn((m, n), generator=g, device="cuda").half()
    T, DL, w = t.arange(m, device="cuda"), t.ones(m, device="cuda"), t.ones(d, device="cuda")
    q = k.sketch_act_quant(X)
    _, mean, rstd, _, _ = k.sketch_norm_fwd(X, w)
    _, lse = k.sketch_xent_fwd(X, idx, lut, T, b, gpr)
    calls = [lambda **a: (k.sketch_matmul_bwd(dY, X, idx, lut, b, gpr, need_dx=False, **a)[1],),
             lambda **a: (k.sketch_matmul_bwd_ckpt(dY, *q, idx, lut, b, gpr, need_dx=False, **a)[1],),
             lambda **a: k.sketch_norm_bwd(X, X, w, mean, rstd, need_dx=False, **a)[1:],
             lambda **a: (k.sketch_xent_bwd(X, idx, lut, T, lse, DL, b, gpr, need_dx=False, **a)[1],)]
    for call in calls:
        want = call()
        for shape in {tuple(o.shape) for o in want}:          # memory of those sizes that holds something
            junk = [t.full(shape, 7.0, device="cuda") for _ in range(16)]
            del junk
        got = call(accumulate=True)
        assert all(t.equal(p, q) for p, q in zip(got, want))
    # one output given, the other new
    dw = t.ones(d, device="cuda")
    _, want_w, want_b = k.sketch_norm_bwd(X, X, w, mean, rstd, need_dx=False)
    junk = [t.full((d,), 7.0, device="cuda") for _ in range(16)]
    del junk
    _, got_w, got_b = k.sketch_norm_bwd(X, X, w, mean, rstd, need_dx=False, dw_out=dw, accumulate=True)
    assert got_w is dw and t.equal(dw, want_w + 1.0) and t.equal(got_b, want_b)


def test_accumulate_into_new_outputs_on_another_stream():
    """The zeros of a new output are written on the stream the call runs on."""
    import torch as t

    import lut_sketched_matmul_amd as k
    m, n, d = 40, 96, 128
    idx = t.randint(0, 256, (n, d // 2), device="cuda", dtype=t.uint8)
    lut = t.randn((n, 2, 16), device="cuda").half()
    X, dY = t.randn((m, d), device="cuda").half(), t.randn((m, n), device="cuda").half()
    want = k.sketch_matmul_bwd(dY, X, idx, lut, 4, 2, need_dx=False)[1]
    s = t.cuda.Stream()
    big = t.randn((4096, 4096), device="cuda")
    t.cuda.synchronize()
    for _ in range(4):                                        # the current stream is busy for a while
        big = (big @ big).clamp_(-1.0, 1.0)
    got = k.sketch_matmul_bwd(dY, X, idx, lut, 4, 2, need_dx=False, accumulate=True, stream=s)[1]
    s.synchronize()
    t.cuda.synchronize()
    assert t.equal(got, want)
