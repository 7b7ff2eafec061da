"""Refusals of the checkpoint, norm and cross entropy entry points (CPU: every call fails its host checks)."""
import pytest
import torch

from lut_sketched_matmul_amd import _lib

EINVAL, EUNSUP, EALIGN, EWS, EALIAS = -1, -2, -3, -4, -6
F32, F16, BF16 = 0, 1, 2
BIG = 1 << 40


def addr(k):
    """Fake 16-byte aligned "device" addresses 16 GiB apart; never dereferenced."""
    return (k + 1) << 34


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def quant(lib, X=addr(0), dt=F16, m=4, d=64, codes=addr(1), scales=addr(2)):
    return lib.sketch_act_quant(X, dt, m, d, codes, scales, None)


def dequant(lib, codes=addr(1), scales=addr(2), m=4, d=64, X=addr(0), dt=F16):
    return lib.sketch_act_dequant(codes, scales, m, d, X, dt, None)


@pytest.mark.parametrize("call", [quant, dequant])
def test_checkpoint_refusals(lib, call):
    assert call(lib, d=0) == EINVAL and call(lib, d=16) == EINVAL and call(lib, d=48) == EINVAL
    assert call(lib, m=-1) == EINVAL
    assert call(lib, m=1 << 20, d=(1 << 14) + 32) == EINVAL   # m * d over 2^34
    assert call(lib, dt=3) == EUNSUP
    assert call(lib, X=None) == EINVAL and call(lib, codes=None) == EINVAL and call(lib, scales=None) == EINVAL
    assert call(lib, X=addr(0) + 8) == EALIGN and call(lib, codes=addr(1) + 4) == EALIGN
    assert call(lib, scales=addr(2) + 1) == EALIGN
    assert call(lib, codes=addr(0) + 256) == EALIAS and call(lib, scales=addr(0)) == EALIAS
    assert call(lib, m=0, X=None, codes=None, scales=None) == 0
    assert quant(lib, scales=addr(1) + 16) == EALIAS


def bwd(lib, dY=addr(0), codes=addr(1), scales=addr(2), dt=F16, idx=addr(3), lut=addr(4), ldt=F16, m=4, n=64, d=512,
        b=4, gpr=2, dX=addr(5), dL=addr(6), acc=0, ws=addr(7), wsb=BIG):
    return lib.sketch_matmul_bwd_ckpt(dY, codes, scales, dt, idx, lut, ldt, m, n, d, b, gpr, dX, dL, acc, ws, wsb, None)


def test_bwd_ckpt_refusals(lib):
    assert bwd(lib, b=5) == EINVAL and bwd(lib, gpr=3) == EINVAL and bwd(lib, acc=2) == EINVAL
    assert bwd(lib, dt=F32) == EUNSUP and bwd(lib, dt=9) == EUNSUP
    for k in ("dY", "codes", "scales", "idx", "lut"):
        assert bwd(lib, **{k: None}) == EINVAL, k
    for k in ("dY", "codes", "scales", "idx", "lut", "dX", "dL", "ws"):
        assert bwd(lib, **{k: addr(9) + 8}) == EALIGN, k
    need = _lib.sketch_matmul_bwd_ckpt_workspace(4, 64, 512, 4, 2, F16, F16)
    assert need >= 4 * 512 * 2
    assert bwd(lib, wsb=need - 1) == EWS and bwd(lib, ws=None) == EWS
    for out in ("dX", "dL", "ws"):
        for k in range(5):
            assert bwd(lib, **{out: addr(k)}) == EALIAS, (out, k)
    assert bwd(lib, dL=addr(5)) == EALIAS and bwd(lib, ws=addr(6)) == EALIAS
    # without dLUT no checkpoint is read, without either output nothing is done
    less = _lib.sketch_matmul_bwd_ckpt_workspace(4, 6400, 512, 4, 2, BF16, F16, need_dlut=False)
    assert 0 < less < _lib.sketch_matmul_bwd_ckpt_workspace(4, 6400, 512, 4, 2, BF16, F16)
    assert bwd(lib, dt=BF16, n=6400, dL=None, codes=None, scales=None, wsb=less - 1) == EWS
    assert bwd(lib, dL=None, codes=None, scales=None, dY=None) == EINVAL
    assert bwd(lib, dX=None, dL=None) == 0 and bwd(lib, m=0, acc=1, dY=None, codes=None, scales=None) == 0


def nfwd(lib, X=addr(0), dt=F16, w=addr(1), bias=addr(2), pdt=F32, m=4, d=64, kind=1, eps=1e-5, Y=addr(3),
         mean=addr(4), rstd=addr(5), codes=addr(6), scales=addr(7)):
    return lib.sketch_norm_fwd(X, dt, w, bias, pdt, m, d, kind, eps, Y, mean, rstd, codes, scales, None)


def nbwd(lib, dY=addr(0), dydt=F16, X=addr(1), dt=F16, codes=None, scales=None, w=addr(2), pdt=F32, mean=addr(3),
         rstd=addr(4), m=4, d=64, kind=1, dX=addr(5), dw=addr(6), db=addr(7), acc=0, ws=addr(8), wsb=BIG):
    return lib.sketch_norm_bwd(dY, dydt, X, dt, codes, scales, w, pdt, mean, rstd, m, d, kind, dX, dw, db, acc, ws,
                               wsb, None)


def test_norm_fwd_refusals(lib):
    assert nfwd(lib, d=0) == EINVAL and nfwd(lib, d=65537) == EINVAL and nfwd(lib, m=-1) == EINVAL
    assert nfwd(lib, m=1 << 31) == EINVAL and nfwd(lib, kind=2) == EINVAL
    assert nfwd(lib, eps=-1.0) == EINVAL and nfwd(lib, eps=float("nan")) == EINVAL
    assert nfwd(lib, dt=5) == EUNSUP and nfwd(lib, pdt=BF16) == EUNSUP
    assert nfwd(lib, d=40) == EINVAL                           # a checkpoint of rows that are not whole blocks
    assert nfwd(lib, scales=None) == EINVAL and nfwd(lib, codes=None) == EINVAL
    for k in ("X", "Y", "mean", "rstd"):
        assert nfwd(lib, **{k: None}) == EINVAL, k
    for k in ("X", "w", "bias", "Y", "mean", "rstd", "codes", "scales"):
        assert nfwd(lib, **{k: addr(9) + 4}) == EALIGN, k
    for k in ("Y", "mean", "rstd", "codes", "scales"):
        for i in range(3):
            assert nfwd(lib, **{k: addr(i)}) == EALIAS, (k, i)
    assert nfwd(lib, mean=addr(3)) == EALIAS and nfwd(lib, scales=addr(6)) == EALIAS
    assert nfwd(lib, m=0, X=None, Y=None, mean=None, rstd=None) == 0


def test_norm_bwd_refusals(lib):
    assert nbwd(lib, d=0) == EINVAL and nbwd(lib, kind=-1) == EINVAL and nbwd(lib, acc=3) == EINVAL
    assert nbwd(lib, dydt=BF16) == EUNSUP and nbwd(lib, pdt=BF16) == EUNSUP
    assert nbwd(lib, X=None) == EINVAL                         # no form of X
    assert nbwd(lib, codes=addr(9), scales=addr(10)) == EINVAL  # both forms
    assert nbwd(lib, X=None, codes=addr(9)) == EINVAL
    assert nbwd(lib, X=None, codes=addr(9), scales=addr(10), d=40) == EINVAL
    for k in ("dY", "mean", "rstd"):
        assert nbwd(lib, **{k: None}) == EINVAL, k
    for k in ("dY", "X", "w", "mean", "rstd", "dX", "dw", "db", "ws"):
        assert nbwd(lib, **{k: addr(9) + 8}) == EALIGN, k
    need = _lib.sketch_norm_bwd_workspace(4, 64)
    assert nbwd(lib, wsb=need - 1) == EWS and nbwd(lib, ws=None) == EWS
    for k in ("dX", "dw", "db", "ws"):
        for i in range(5):
            assert nbwd(lib, **{k: addr(i)}) == EALIAS, (k, i)
    assert nbwd(lib, dw=addr(5)) == EALIAS and nbwd(lib, ws=addr(7)) == EALIAS
    assert nbwd(lib, dX=None, dw=None, db=None) == 0           # nothing asked for
    assert nbwd(lib, m=0, acc=1, dY=None, X=None) == 0


def xf(lib, X=addr(0), dt=F16, idx=addr(1), lut=addr(2), ldt=F16, t=addr(3), ign=-100, m=4, n=100, d=64, b=4, gpr=2,
       loss=addr(4), lse=addr(5), ws=addr(6), wsb=BIG):
    return lib.sketch_xent_fwd(X, dt, idx, lut, ldt, t, ign, m, n, d, b, gpr, loss, lse, ws, wsb, None)


def xb(lib, X=addr(0), dt=F16, idx=addr(1), lut=addr(2), ldt=F16, t=addr(3), ign=-100, lse=addr(4), dl=addr(5), m=4,
       n=100, d=64, b=4, gpr=2, dX=addr(6), dL=addr(7), acc=0, ws=addr(8), wsb=BIG):
    return lib.sketch_xent_bwd(X, dt, idx, lut, ldt, t, ign, lse, dl, m, n, d, b, gpr, dX, dL, acc, ws, wsb, None)


@pytest.mark.parametrize("call", [xf, xb])
def test_xent_shape_and_dtype_refusals(lib, call):
    assert call(lib, n=0) == EINVAL and call(lib, b=1) == EINVAL and call(lib, m=-1) == EINVAL
    assert call(lib, gpr=4) == EINVAL                          # groups of 16 columns
    assert call(lib, m=(1 << 22) + 1) == EINVAL and call(lib, d=(1 << 20) + 64) == EINVAL
    assert call(lib, m=1 << 22, n=1 << 17) == EINVAL           # 2^14 x 2^9 tiles
    assert call(lib, n=1 << 30, gpr=2) == EINVAL
    for pair in ((F32, F32), (F16, BF16), (F32, F16), (F16, F32), (7, F16)):
        assert call(lib, dt=pair[0], ldt=pair[1]) == EUNSUP, pair


def test_xent_buffer_refusals(lib):
    for k in ("X", "idx", "lut", "t", "loss", "lse"):
        assert xf(lib, **{k: None}) == EINVAL, k
    for k in ("X", "idx", "lut", "loss", "lse", "ws"):
        assert xf(lib, **{k: addr(9) + 8}) == EALIGN, k
    assert xf(lib, t=addr(3) + 4) == EALIGN
    for k in ("loss", "lse", "ws"):
        for i in range(4):
            assert xf(lib, **{k: addr(i)}) == EALIAS, (k, i)
    assert xf(lib, lse=addr(4)) == EALIAS and xf(lib, ws=addr(5)) == EALIAS
    need = _lib.sketch_xent_fwd_workspace(4, 100, 64, 4, 2, F16, F16)
    assert need > 0 and xf(lib, wsb=need - 1) == EWS and xf(lib, ws=None) == EWS
    assert xf(lib, m=0, X=None, t=None, loss=None, lse=None, ws=None, wsb=0) == 0

    for k in ("X", "idx", "lut", "t", "lse", "dl"):
        assert xb(lib, **{k: None}) == EINVAL, k
    for k in ("X", "idx", "lut", "lse", "dl", "dX", "dL", "ws"):
        assert xb(lib, **{k: addr(9) + 8}) == EALIGN, k
    for k in ("dX", "dL", "ws"):
        for i in range(6):
            assert xb(lib, **{k: addr(i)}) == EALIAS, (k, i)
    assert xb(lib, dL=addr(6)) == EALIAS and xb(lib, acc=2) == EINVAL
    need = _lib.sketch_xent_bwd_workspace(4, 100, 64, 4, 2, F16, F16)
    assert need > 0 and xb(lib, wsb=need - 1) == EWS
    less = _lib.sketch_xent_bwd_workspace(4, 100, 64, 4, 2, F16, F16, need_dlut=False)
    assert 0 < less < need and xb(lib, dL=None, wsb=less - 1) == EWS
    assert xb(lib, dX=None, dL=None) == 0
    assert xb(lib, m=0, acc=1, X=None, t=None, lse=None, dl=None) == 0


def test_xent_mean_refusals(lib):
    call = lambda loss=addr(0), t=addr(1), m=4, mean=addr(2), w=addr(3): lib.sketch_xent_mean(loss, t, -100, m, mean, w,
                                                                                              None)
    assert call(m=0) == EINVAL and call(m=1 << 31) == EINVAL
    for k in ("loss", "t", "mean", "w"):
        assert call(**{k: None}) == EINVAL, k
    assert call(loss=addr(0) + 8) == EALIGN and call(w=addr(3) + 4) == EALIGN and call(t=addr(1) + 4) == EALIGN
    assert call(mean=addr(2) + 2) == EALIGN
    for k in ("mean", "w"):
        assert call(**{k: addr(0)}) == EALIAS and call(**{k: addr(1)}) == EALIAS
    assert call(mean=addr(3) + 12) == EALIAS


def test_wrappers_check_tensors_before_the_call():
    X = torch.zeros(4, 64, dtype=torch.float16)
    codes, scales = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        _lib.sketch_act_quant(X)
    with pytest.raises(ValueError, match="blocks of 32"):
        _lib.sketch_act_quant(X[:, :48].contiguous())
    with pytest.raises(ValueError, match="codes"):
        _lib.sketch_act_quant(X, codes=codes[:3])
    with pytest.raises(TypeError, match="scales"):
        _lib.sketch_act_quant(X, scales=scales.to(torch.int32))
    with pytest.raises(ValueError, match="scales"):
        _lib.sketch_act_dequant(codes, scales[:, :1], torch.float16)
    with pytest.raises(TypeError, match="dtype"):
        _lib.sketch_act_dequant(codes, scales, torch.float64)
    with pytest.raises(TypeError, match="out"):
        _lib.sketch_act_dequant(codes, scales, torch.float16, out=X.float())
    idx, lut = torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 2, 16, dtype=torch.float16)
    dY = torch.zeros(4, 16, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        _lib.sketch_matmul_bwd_ckpt(dY, codes, scales, idx, lut, 4, 2)
    with pytest.raises(ValueError, match="codes"):
        _lib.sketch_matmul_bwd_ckpt(dY, codes[:3], scales, idx, lut, 4, 2)
    with pytest.raises(TypeError, match="codes"):
        _lib.sketch_matmul_bwd_ckpt(dY, codes.to(torch.uint8), scales, idx, lut, 4, 2)
    w = torch.zeros(64)
    with pytest.raises(ValueError, match="kind"):
        _lib.sketch_norm_fwd(X, w, kind="batch")
    with pytest.raises(ValueError, match="weight"):
        _lib.sketch_norm_fwd(X, w[:63])
    with pytest.raises(TypeError, match="weight"):
        _lib.sketch_norm_fwd(X, w.to(torch.bfloat16))
    with pytest.raises(TypeError, match="one dtype"):
        _lib.sketch_norm_fwd(X, w, w.to(torch.float16))
    with pytest.raises(ValueError, match="blocks of 32"):
        _lib.sketch_norm_fwd(X[:, :40].contiguous(), checkpoint=True)
    with pytest.raises(ValueError, match="mean"):
        _lib.sketch_norm_bwd(X, X, w, None, torch.zeros(4))
    with pytest.raises(TypeError, match="dY"):
        _lib.sketch_norm_bwd(X.to(torch.bfloat16), X, w, torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError, match="rstd"):
        _lib.sketch_norm_bwd(X, X, w, torch.zeros(4), torch.zeros(3))
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        _lib.sketch_xent_fwd(X, idx, lut, t, 4, 2)
    with pytest.raises(TypeError, match="targets"):
        _lib.sketch_xent_fwd(X, idx, lut, t.int(), 4, 2)
    with pytest.raises(ValueError, match="targets"):
        _lib.sketch_xent_fwd(X, idx, lut, t[:3], 4, 2)
    with pytest.raises(TypeError, match="X"):
        _lib.sketch_xent_fwd(X.float(), idx, lut, t, 4, 2)
    with pytest.raises(ValueError, match="lse"):
        _lib.sketch_xent_bwd(X, idx, lut, t, torch.zeros(3), torch.zeros(4), 4, 2)
    with pytest.raises(TypeError, match="dloss"):
        _lib.sketch_xent_bwd(X, idx, lut, t, torch.zeros(4), torch.zeros(4, dtype=torch.float16), 4, 2)


def test_bwd_ckpt_of_more_rows_than_a_launch_takes(lib):
    """2^22 blocks of 128 weight rows x a group, 512 threads each, is what one launch of the table gradient takes."""
    most = (1 << 29) // 2
    assert bwd(lib, m=1, n=most + 1) == EINVAL and bwd(lib, m=1, n=1 << 31, gpr=1, d=32) == EINVAL
    assert bwd(lib, m=1, n=most, ws=None) == EWS
    assert _lib.sketch_matmul_bwd_ckpt_workspace(1, most + 1, 512, 4, 2, F16, F16) == 0


@pytest.mark.parametrize("m,n,dt,need,forms", [
    (4096, 128256, BF16, (True, False), 1), (4096, 128256, F16, (True, True), 2), (4096, 128256, BF16, (True, True), 3),
    (1 << 22, 512, F16, (True, False), 1), (1 << 22, 512, F16, (False, True), 2), (1 << 22, 512, BF16, (True, True), 3),
])
def test_xent_bwd_workspace_is_as_stated(m, n, dt, need, forms):
    """dZ: 256 MiB, or 512 bytes per token and form; beside it the other terms of the header, d = 32 columns."""
    d, gpr = 32, 1
    got = _lib.sketch_xent_bwd_workspace(m, n, d, 4, gpr, dt, F16, *need)
    tiles = m // 256
    dx = max(2, 512 // tiles) * m * d * 4 if need[0] else 0
    tables = 64 * n * gpr * 16 * 4 if need[1] else 0                 # partial tables, when the row blocks are few
    vectors = 6 * (m * 4 + 256)
    assert got <= max(1 << 28, 512 * m * forms) + dx + 2 * (2 * m * d + 256) + tables + vectors
    assert got >= min(1 << 28, 512 * m * forms) // 2
