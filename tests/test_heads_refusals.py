"""Refusals of dropout, the adapters and head rotation (CPU: every call fails its host checks, or is empty)."""
import pytest
import torch

import lut_sketched_matmul_amd as skm
from lut_sketched_matmul_amd import _lib

EINVAL, EUNSUP, EALIGN, EWS, EALIAS = -1, -2, -3, -4, -6
F32, F16, BF16 = 0, 1, 2
BIG = 1 << 40
NAN = float("nan")


def addr(k):
    """Fake 16-byte aligned "device" addresses 64 GiB apart; never dereferenced."""
    return (k + 1) << 36


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def drop(lib, X=addr(0), dt=BF16, res=addr(1), count=100, p=0.1, seed=addr(2), Y=addr(3)):
    return lib.sketch_dropout(X, dt, res, count, p, seed, Y, None)


def test_dropout_refusals(lib):
    assert drop(lib, count=-1) == EINVAL and drop(lib, count=(1 << 40) + 1) == EINVAL
    assert drop(lib, p=-0.01) == EINVAL and drop(lib, p=1.01) == EINVAL and drop(lib, p=NAN) == EINVAL
    assert drop(lib, dt=3) == EUNSUP
    assert drop(lib, X=None) == EINVAL and drop(lib, Y=None) == EINVAL and drop(lib, seed=None) == EINVAL
    for k in ("X", "res", "Y"):
        assert drop(lib, **{k: addr(9) + 8}) == EALIGN
    assert drop(lib, seed=addr(2) + 4) == EALIGN
    assert drop(lib, Y=addr(0)) == EALIAS and drop(lib, Y=addr(1) + 16) == EALIAS and drop(lib, Y=addr(2)) == EALIAS
    assert drop(lib, count=0, X=None, Y=None, res=None, seed=None) == 0


def afwd(lib, X=addr(0), A=addr(1), B=addr(2), dt=BF16, ids=addr(3), S=3, scale=addr(4), base=addr(5), p=0.1,
         seed=addr(6), m=40, n=50, d=64, r=8, Y=addr(7), H=addr(8), ws=addr(9), wsb=BIG):
    return lib.sketch_adapter_fwd(X, A, B, dt, ids, S, scale, base, p, seed, m, n, d, r, Y, H, ws, wsb, None)


def abwd(lib, dY=addr(10), X=addr(0), H=addr(8), A=addr(1), B=addr(2), dt=BF16, ids=addr(3), S=3, scale=addr(4),
         base=addr(5), p=0.1, seed=addr(6), m=40, n=50, d=64, r=8, dX=addr(7), dA=addr(11), dB=addr(12), acc=0,
         ws=addr(9), wsb=BIG):
    return lib.sketch_adapter_bwd(dY, X, H, A, B, dt, ids, S, scale, base, p, seed, m, n, d, r, dX, dA, dB, acc, ws,
                                  wsb, None)


@pytest.mark.parametrize("call", [afwd, abwd])
def test_adapter_refusals(lib, call):
    for bad in (dict(m=-1), dict(m=(1 << 22) + 1), dict(n=0), dict(n=(1 << 24) + 1), dict(d=0), dict(d=48),
                dict(d=(1 << 20) + 32), dict(r=0), dict(r=129), dict(S=0), dict(m=1 << 22, n=4097),
                dict(m=1 << 22, d=4128), dict(p=-0.1), dict(p=1.5), dict(p=NAN)):
        assert call(lib, **bad) == EINVAL, bad
    assert call(lib, dt=F32) == EUNSUP and call(lib, dt=9) == EUNSUP
    for k in ("X", "A", "B", "seed"):
        assert call(lib, **{k: None}) == EINVAL, k
    for k in ("X", "A", "B", "base", "H", "ws"):
        assert call(lib, **{k: addr(14) + 8}) == EALIGN, k
    assert call(lib, ids=addr(14) + 2) == EALIGN and call(lib, scale=addr(14) + 2) == EALIGN
    assert call(lib, seed=addr(14) + 4) == EALIGN and call(lib, ws=None) == EWS
    for k in (0, 1, 2, 3, 4, 6):
        assert call(lib, ws=addr(k)) == EALIAS, k


def test_adapter_forward_refusals(lib):
    assert afwd(lib, S=(1 << 20) + 1) == EINVAL and afwd(lib, Y=None) == EINVAL
    need = skm.sketch_adapter_fwd_workspace(40, 50, 64, 8, 3)
    assert need >= 40 * 8 * 4 and afwd(lib, wsb=need - 1) == EWS
    for o in ("Y", "H"):
        for k in (0, 1, 2, 3, 4, 6, 9):
            assert afwd(lib, **{o: addr(k)}) == EALIAS, (o, k)
    assert afwd(lib, Y=addr(8)) == EALIAS and afwd(lib, H=addr(5)) == EALIAS
    assert afwd(lib, Y=addr(5) + 16) == EALIAS           # over the base, but not the base itself
    assert afwd(lib, m=0, X=None, Y=None, seed=None, ws=None, wsb=0) == 0
    # a few tokens without dropout take none
    assert skm.sketch_adapter_fwd_workspace(40, 50, 64, 8, 3, has_dropout=False) == 0
    assert skm.sketch_adapter_fwd_workspace(400, 50, 64, 8, 3, has_dropout=False) >= 400 * 8 * 4
    assert afwd(lib, m=400, p=0.0, seed=None, wsb=400 * 8 * 4 - 1) == EWS
    assert skm.sketch_adapter_fwd_workspace(40, 50, 48, 8, 3) == 0 and skm.sketch_adapter_fwd_workspace(0, 50, 64, 8, 3) == 0


def test_adapter_backward_refusals(lib):
    assert abwd(lib, S=4097) == EINVAL and abwd(lib, acc=2) == EINVAL
    assert abwd(lib, m=1024, n=1 << 24, S=512) == EINVAL     # more blocks than one launch takes
    assert skm.sketch_adapter_bwd_workspace(1024, 1 << 24, 64, 8, 512) == 0
    assert skm.sketch_adapter_bwd_workspace(1024, 1 << 24, 64, 8, 16) > 0
    assert abwd(lib, dY=None) == EINVAL and abwd(lib, H=None) == EINVAL
    need = skm.sketch_adapter_bwd_workspace(40, 50, 64, 8, 3)
    assert abwd(lib, wsb=need - 1) == EWS
    for o in ("dX", "dA", "dB"):
        assert abwd(lib, **{o: addr(14) + 4}) == EALIGN
        for k in (0, 1, 2, 3, 4, 5, 6, 8, 9, 10):
            assert abwd(lib, **{o: addr(k)}) == EALIAS, (o, k)
    assert abwd(lib, dA=addr(7)) == EALIAS and abwd(lib, dB=addr(11)) == EALIAS
    assert abwd(lib, dX=None, dA=None, dB=None) == 0
    assert abwd(lib, m=0, acc=1, dY=None, X=None, H=None, ws=None, wsb=0) == 0
    # what is not read may be left out, and takes no workspace
    less = skm.sketch_adapter_bwd_workspace(40, 50, 64, 8, 3, need_dx=False, need_da=False)
    assert 0 < less < need
    assert abwd(lib, dX=None, dA=None, X=None, seed=None, wsb=less - 1) == EWS
    assert skm.sketch_adapter_bwd_workspace(40, 50, 64, 8, 3, need_dx=False, need_da=False, need_db=False) == 0


def rfwd(lib, Q=addr(0), ldq=512, hq=4, K=addr(1), ldk=256, hk=2, dt=BF16, pos=addr(2), freq=addr(3), qw=addr(4),
         kw=addr(5), m=10, dh=128, rot=128, pairs=0, norm=1, eps=1e-6, Qo=addr(6), ldqo=512, Ko=addr(7), ldko=256):
    return lib.sketch_rotary_fwd(Q, ldq, hq, K, ldk, hk, dt, pos, freq, qw, kw, m, dh, rot, pairs, norm, eps, Qo, ldqo,
                                 Ko, ldko, None)


def rbwd(lib, dQ=addr(8), lddq=512, hq=4, dK=addr(9), lddk=256, hk=2, dt=BF16, Q=addr(0), ldq=512, K=addr(1), ldk=256,
         pos=addr(2), freq=addr(3), qw=addr(4), kw=addr(5), m=10, dh=128, rot=128, pairs=0, norm=1, eps=1e-6, Qo=addr(6),
         ldqo=512, Ko=addr(7), ldko=256, dqw=addr(10), dkw=addr(11), acc=0, ws=addr(12), wsb=BIG):
    return lib.sketch_rotary_bwd(dQ, lddq, hq, dK, lddk, hk, dt, Q, ldq, K, ldk, pos, freq, qw, kw, m, dh, rot, pairs,
                                 norm, eps, Qo, ldqo, Ko, ldko, dqw, dkw, acc, ws, wsb, None)


@pytest.mark.parametrize("call", [rfwd, rbwd])
def test_rotary_refusals(lib, call):
    for bad in (dict(m=-1), dict(m=1 << 31), dict(hq=0), dict(hk=-1), dict(hq=65537), dict(dh=0), dict(dh=127),
                dict(dh=1026, ldq=5000), dict(rot=0), dict(rot=63), dict(rot=130), dict(pairs=2), dict(norm=2),
                dict(eps=-1.0), dict(eps=NAN), dict(Q=None), dict(K=None), dict(pos=None), dict(freq=None),
                dict(Qo=None), dict(Ko=None), dict(ldq=511), dict(ldk=255), dict(ldqo=511), dict(ldko=255),
                dict(ldq=1 << 40)):
        assert call(lib, **bad) == EINVAL, bad
    assert call(lib, dt=3) == EUNSUP
    assert call(lib, Q=addr(0) + 1) == EALIGN and call(lib, dt=F32, Ko=addr(7) + 2) == EALIGN
    assert call(lib, pos=addr(2) + 4) == EALIGN and call(lib, freq=addr(3) + 4) == EALIGN
    assert call(lib, qw=addr(4) + 4) == EALIGN and call(lib, kw=addr(5) + 8) == EALIGN
    for k in (2, 3, 4, 5):
        assert call(lib, Qo=addr(k)) == EALIAS and call(lib, Ko=addr(k) + 64) == EALIAS, k
    assert call(lib, Qo=addr(1)) == EALIAS and call(lib, Ko=addr(0)) == EALIAS and call(lib, Ko=addr(6)) == EALIAS
    # outputs in one joined buffer: columns beside each other are fine, shared ones are not
    assert call(lib, Qo=addr(6), ldqo=768, Ko=addr(6) + 1022, ldko=768) == EALIAS
    assert call(lib, Qo=addr(6), ldqo=768, Ko=addr(6) + 1024, ldko=700) == EALIAS
    assert call(lib, Qo=addr(6), ldqo=768, Ko=addr(6) + 1026, ldko=768) == EALIAS   # its end reaches the next row


def test_rotary_forward_refusals(lib):
    assert rfwd(lib, Qo=addr(0) + 2) == EALIAS and rfwd(lib, Qo=addr(0), ldqo=600) == EALIAS
    assert rfwd(lib, m=0, Q=None, K=None, pos=None, freq=None, Qo=None, Ko=None) == 0


def test_rotary_backward_refusals(lib):
    assert rbwd(lib, acc=3) == EINVAL and rbwd(lib, norm=0) == EINVAL     # weight gradients without a norm
    assert rbwd(lib, dQ=None) == EINVAL and rbwd(lib, lddk=255) == EINVAL
    need = skm.sketch_rotary_bwd_workspace(128)
    assert need > 0 and rbwd(lib, wsb=need - 1) == EWS and rbwd(lib, ws=None) == EWS
    assert rbwd(lib, Qo=addr(0)) == EALIAS and rbwd(lib, Qo=addr(8)) == EALIAS and rbwd(lib, Ko=addr(9)) == EALIAS
    for k in (2, 3, 4, 5, 0, 1, 8, 9, 6, 7):
        assert rbwd(lib, dqw=addr(k)) == EALIAS and rbwd(lib, ws=addr(k)) == EALIAS, k
    assert rbwd(lib, dkw=addr(10)) == EALIAS and rbwd(lib, dqw=addr(10) + 4) == EALIGN
    assert rbwd(lib, m=0, acc=1, dQ=None, dK=None) == 0


class OnGpu(torch.Tensor):
    """A CPU tensor that says it lives on a GPU: the bindings' shape and dtype checks come before any launch."""

    @property
    def is_cuda(self):
        return True


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


def test_binding_checks():
    f32, f64, i32, i64 = torch.float32, torch.float64, torch.int32, torch.int64
    X, A, B, seed = t(4, 64), t(2, 8, 64), t(2, 10, 8), t(2, dtype=i64)
    with pytest.raises(ValueError):
        skm.sketch_dropout(X, 1.5, seed)
    with pytest.raises(ValueError):
        skm.sketch_dropout(X, 0.5)                            # no seed
    with pytest.raises(ValueError):
        skm.sketch_dropout(X, 0.5, t(3, dtype=i64))
    with pytest.raises(TypeError):
        skm.sketch_dropout(X, 0.5, t(2, dtype=i32))
    with pytest.raises(ValueError):
        skm.sketch_dropout(X, 0.5, seed, residual=t(4, 65))
    with pytest.raises(TypeError):
        skm.sketch_dropout(X, 0.5, seed, residual=t(4, 64, dtype=f32))
    for bad, kind in ((dict(A=t(2, 8, 32)), ValueError), (dict(B=t(3, 10, 8)), ValueError), (dict(B=t(2, 10, 9)), ValueError),
                      (dict(A=t(8, 64)), ValueError), (dict(A=t(2, 8, 64, dtype=torch.float16)), TypeError),
                      (dict(X=t(4, 64, dtype=f32)), TypeError), (dict(base=t(4, 11)), ValueError),
                      (dict(adapter=t(5, dtype=i32)), ValueError), (dict(adapter=t(4, dtype=i64)), TypeError),
                      (dict(scale=t(3, dtype=f32)), ValueError), (dict(p=0.5), ValueError), (dict(out=t(4, 9)), ValueError)):
        a = dict(X=X, A=A, B=B)
        a.update(bad)
        with pytest.raises(kind):
            skm.sketch_adapter_fwd(**a)
    dY, H = t(4, 10), t(4, 8, dtype=f32)
    for bad, kind in ((dict(dY=t(4, 9)), ValueError), (dict(H=None), ValueError), (dict(H=t(4, 8)), TypeError),
                      (dict(base_dx=t(4, 64)), TypeError), (dict(da_out=t(2, 8, 63, dtype=f32)), ValueError),
                      (dict(db_out=t(2, 10, 8)), TypeError)):
        a = dict(dY=dY, X=X, H=H, A=A, B=B)
        a.update(bad)
        with pytest.raises(kind):
            skm.sketch_adapter_bwd(**a)
    q, k, pos, f, w = t(4, 8, 64), t(4, 2, 64), t(4, dtype=i64), t(32, dtype=f64), t(64, dtype=f32)
    for bad, kind in ((dict(q=t(4, 64)), ValueError), (dict(k=t(4, 2, 32)), ValueError), (dict(k=t(3, 2, 64)), ValueError),
                      (dict(k=t(4, 2, 64, dtype=f32)), TypeError), (dict(positions=t(4, dtype=i32)), TypeError),
                      (dict(positions=t(5, dtype=i64)), ValueError), (dict(inv_freq=t(32, dtype=f32)), TypeError),
                      (dict(inv_freq=t(33, dtype=f64)), ValueError), (dict(inv_freq=t(0, dtype=f64)), ValueError),
                      (dict(q_weight=w), ValueError), (dict(eps=1e-6, q_weight=t(64)), TypeError),
                      (dict(eps=1e-6, q_weight=t(32, dtype=f32)), ValueError), (dict(pairs="odd"), ValueError),
                      (dict(q=t(4, 64, 8).transpose(1, 2)), ValueError), (dict(q=t(1, 8, 64).expand(4, 8, 64)), ValueError),
                      (dict(k=None, k_out=k), ValueError)):
        a = dict(q=q, k=k, positions=pos, inv_freq=f)
        a.update(bad)
        with pytest.raises(kind):
            skm.sketch_rotary_fwd(**a)
    for bad, kind in ((dict(dq=t(4, 8, 32)), ValueError), (dict(dk=None), ValueError),
                      (dict(dk=t(4, 2, 64, dtype=f32)), TypeError),
                      (dict(qw_out=w), ValueError), (dict(eps=1e-6, qw_out=t(64)), TypeError)):
        a = dict(dq=q, dk=k, q=q, k=k, positions=pos, inv_freq=f)
        a.update(bad)
        with pytest.raises(kind):
            skm.sketch_rotary_bwd(**a)
    with pytest.raises(ValueError):
        skm.sketch_dropout(torch.zeros(8), 0.0)               # not on the GPU


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("m,n,d,r,S,word", [(5, 64, 64, 1, 4097, "4096"), (1024, 1 << 24, 64, 8, 512, "2\\^24")])
def test_adapter_backward_names_its_limits(m, n, d, r, S, word):
    """What the forward takes and the backward does not is refused with the reason, not with a bare status."""
    args = (meta(m, n), meta(m, d), meta(m, r, dtype=torch.float32), meta(S, r, d), meta(S, n, r))
    with pytest.raises(ValueError, match=word):
        skm.sketch_adapter_bwd(*args)
    with pytest.raises(ValueError, match="GPU"):  # (in range: the next check's)
        skm.sketch_adapter_bwd(meta(m, 64), args[1], args[2], meta(4, r, d), meta(4, 64, r))
