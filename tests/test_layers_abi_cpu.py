"""Refusals of the layer operators that need no GPU: the C entry points check their
arguments before any HIP call, the binding checks tensors before it calls them."""
import ctypes
import os

import pytest
import torch

import fp64_gemm_emulation_ozk_amd as ozk

OK, EINVAL, EWORKSPACE, ERANGE, EHIP, EUNSUPPORTED = 0, -1, -2, -3, -4, -5
FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: every call below fails validation
ODD = ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ozk.LIB_PATH):
        from fp64_gemm_emulation_ozk_amd.build import build_library
        build_library(verbose=False)
    return ozk.library()


def _caller(f, names, defaults):
    def call(**kw):
        args = dict(defaults, **kw)
        assert set(kw) <= set(names)
        return f(*[args[n] for n in names])
    return call


def test_dgemm_epilogue_refusals(lib):
    names = "m n k A lda B ldb bias act R ldr Z ldz C ldc r scaling ws wsb stream".split()
    call = _caller(lib.ozk_dgemm_epilogue, names, dict(
        m=4, n=4, k=4, A=FAKE, lda=4, B=FAKE, ldb=4, bias=FAKE, act=2, R=FAKE, ldr=4, Z=FAKE,
        ldz=4, C=FAKE, ldc=4, r=14, scaling=0, ws=FAKE, wsb=1 << 20, stream=None))
    for bad in (dict(act=-1), dict(act=5), dict(r=0), dict(r=21), dict(scaling=2), dict(m=-1),
                dict(k=0), dict(lda=3), dict(ldb=3), dict(ldc=3), dict(ldr=3), dict(ldz=3),
                dict(A=None), dict(B=None), dict(C=None), dict(ws=ODD)):
        assert call(**bad) == EINVAL, bad
    assert call(k=131072, lda=131072) == ERANGE
    assert call(r=2, k=1 << 16, lda=1 << 16) == ERANGE          # no bit budget
    assert call(ws=None, wsb=0) == EWORKSPACE and call(wsb=16) == EWORKSPACE
    assert call(m=0, ws=None, wsb=0) == OK and call(n=0, ws=None, wsb=0) == OK
    out = ctypes.c_size_t()
    size = lib.ozk_dgemm_epilogue_workspace_size
    assert size(4, 4, 4, 14, None) == EINVAL and size(4, 4, 0, 14, ctypes.byref(out)) == EINVAL
    assert size(4, 4, 131072, 14, ctypes.byref(out)) == ERANGE
    assert size(4, 4, 4, 14, ctypes.byref(out)) == OK
    assert call(wsb=out.value - 1) == EWORKSPACE
    # absent operands ask for nothing of their leading dimensions
    assert call(R=None, ldr=0, Z=None, ldz=0, wsb=16) == EWORKSPACE


def test_dgemm_epilogue_grad_refusals(lib):
    names = "m n k dC lddc A lda B ldb Z ldz act dA ldda dB lddb db r scaling ws wsb stream".split()
    call = _caller(lib.ozk_dgemm_epilogue_grad, names, dict(
        m=4, n=4, k=4, dC=FAKE, lddc=4, A=FAKE, lda=4, B=FAKE, ldb=4, Z=FAKE, ldz=4, act=1,
        dA=FAKE, ldda=4, dB=FAKE, lddb=4, db=FAKE, r=14, scaling=1, ws=FAKE, wsb=1 << 30,
        stream=None))
    for bad in (dict(act=5), dict(r=0), dict(scaling=-1), dict(n=-1), dict(k=0), dict(lddc=3),
                dict(ldz=3), dict(ldda=3), dict(lddb=3), dict(lda=3), dict(ldb=3),
                dict(dC=None), dict(Z=None), dict(A=None), dict(B=None), dict(ws=ODD)):
        assert call(**bad) == EINVAL, bad
    assert call(m=131072) == ERANGE and call(n=131072) == ERANGE and call(k=131072) == ERANGE
    assert call(r=2, m=1 << 16, scaling=0) == ERANGE            # dB's budget
    assert call(ws=None, wsb=0) == EWORKSPACE and call(wsb=256) == EWORKSPACE
    assert call(dA=None, dB=None, db=None, ws=None, wsb=0) == OK
    assert call(m=0, dB=None, db=None, ws=None, wsb=0) == OK    # dA has no rows
    out = ctypes.c_size_t()
    size = lib.ozk_dgemm_epilogue_grad_workspace_size
    assert size(4, 4, 4, 14, None) == EINVAL and size(4, 4, 4, 0, ctypes.byref(out)) == EINVAL
    assert size(131072, 4, 4, 14, ctypes.byref(out)) == ERANGE
    assert size(64, 96, 32, 14, ctypes.byref(out)) == OK
    assert out.value >= 8 * 64 * 96 + 14 * (64 + 32) * 128 + 14 * 64 * 32


def test_int8linear_refusals(lib):
    names = "m n k X ldx sx W ldw sw bias act R ldr type C ldc ws wsb stream".split()
    call = _caller(lib.ozk_int8linear, names, dict(
        m=4, n=4, k=4, X=FAKE, ldx=4, sx=FAKE, W=FAKE, ldw=4, sw=FAKE, bias=FAKE, act=0, R=FAKE,
        ldr=4, type=3, C=FAKE, ldc=4, ws=FAKE, wsb=0, stream=None))
    for bad in (dict(act=5), dict(act=-1), dict(type=0), dict(type=4), dict(type=-1), dict(m=-1),
                dict(n=-1), dict(k=0), dict(ldx=3), dict(ldw=3), dict(ldc=3), dict(ldr=3),
                dict(X=None), dict(W=None), dict(sx=None), dict(sw=None), dict(C=None),
                dict(sx=ODD), dict(sw=ODD), dict(bias=ODD), dict(R=ODD), dict(C=ODD)):
        assert call(**bad) == EINVAL, bad
    assert call(k=131072, ldx=131072, ldw=131072) == ERANGE
    assert call(m=1 << 31) == EUNSUPPORTED
    assert call(m=0) == OK and call(n=0) == OK
    # a shape whose K is split over workgroups needs its partial sums, unaligned operands of
    # more than a few rows an aligned copy; a call is held to what its own operands need
    for m, n, k, aligned in ((1, 16, 131071, False), (100, 100, 100, False),
                             (100, 100, 8192, True)):
        need = ozk.ozk_int8linear_workspace_size(m, n, k, aligned)
        assert need > 0
        big = dict(m=m, n=n, k=k, ldx=k, ldw=k, ldc=n, ldr=n)
        assert call(**big) == EWORKSPACE and call(**big, wsb=need - 1) == EWORKSPACE
        assert call(**big, wsb=need, ws=None) == EWORKSPACE
        assert call(**big, wsb=need, ws=ODD) == EINVAL
        if aligned:
            assert ozk.ozk_int8linear_workspace_size(m, n, k, False) >= need + (m + n) * k
            assert call(**big, wsb=need, X=ctypes.c_void_p(0x1008)) == EWORKSPACE
    assert ozk.ozk_int8linear_workspace_size(100, 4096, 128, True) == 0   # one K step
    out = ctypes.c_size_t()
    size = lib.ozk_int8linear_workspace_size
    assert size(4, 4, 0, 0, ctypes.byref(out)) == EINVAL and size(4, 4, 4, 0, None) == EINVAL
    assert size(4, 4, 4, 2, ctypes.byref(out)) == EINVAL
    assert size(4, 4, 131072, 0, ctypes.byref(out)) == ERANGE


@pytest.mark.parametrize("m", [1, 16, 17, 31, 32, 33, 64, 65, 100, 300, 1000])
def test_int8linear_general_query_serves_aligned_operands(lib, m):
    """aligned = 0 stands for any operands: its size is enough for those that are aligned, which
    run in another way (17 to 64 rows most of all)."""
    names = "m n k X ldx sx W ldw sw bias act R ldr type C ldc ws wsb stream".split()
    call = _caller(lib.ozk_int8linear, names, dict(
        m=m, n=4, k=4, X=FAKE, ldx=4, sx=FAKE, W=FAKE, ldw=4, sw=FAKE, bias=None, act=0, R=None,
        ldr=0, type=3, C=FAKE, ldc=4, ws=None, wsb=0, stream=None))
    size = ozk.ozk_int8linear_workspace_size
    for n in (1, 16, 33, 256, 1000, 4096, 8192):
        for k in (16, 128, 1024, 4096, 16384, 131056):
            general, tiled = size(m, n, k), size(m, n, k, True)
            assert general >= tiled, (m, n, k)
            if tiled:   # it is taken as enough: only the workspace's address is refused
                assert call(n=n, k=k, ldx=k, ldw=k, ldc=n, ws=ODD, wsb=general) == EINVAL
            # a K that no operand can be aligned for
            assert size(m, n, k + 1) == size(m, n, k + 1, True)


def test_int8linear_refuses_what_a_launch_cannot_take(lib):
    """2^32 threads and more, found before any HIP call."""
    names = "m n k X ldx sx W ldw sw bias act R ldr type C ldc ws wsb stream".split()
    call = _caller(lib.ozk_int8linear, names, dict(
        m=4, n=4, k=16, X=FAKE, ldx=16, sx=FAKE, W=FAKE, ldw=16, sw=FAKE, bias=None, act=0, R=None,
        ldr=0, type=3, C=FAKE, ldc=1 << 31, ws=FAKE, wsb=1 << 62, stream=None))
    assert call(n=(1 << 27) + 1) == EUNSUPPORTED
    assert call(k=17, ldx=17, ldw=17, n=(1 << 27) + 1) == EUNSUPPORTED
    assert call(m=1 << 20, n=1 << 20) == EUNSUPPORTED
    assert call(m=65, n=1 << 20, k=131071, ldx=131071, ldw=131071) == EUNSUPPORTED


@pytest.mark.parametrize("kind", [0, 1, 2, 3])
def test_row_operator_refusals(lib, kind):
    names = "rows cols type x ldx norm g b eps q ldq scale stream".split()
    call = _caller(lib.ozk_int8quant_rows, names, dict(
        rows=4, cols=4, type=kind, x=FAKE, ldx=4, norm=1, g=FAKE, b=FAKE, eps=1e-5, q=FAKE,
        ldq=4, scale=FAKE, stream=None))
    for bad in (dict(type=4), dict(type=-1), dict(rows=-1), dict(cols=0), dict(ldx=3),
                dict(ldq=3), dict(norm=2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(x=None), dict(q=None), dict(scale=None), dict(x=ODD), dict(g=ODD),
                dict(b=ODD), dict(scale=ODD), dict(norm=0)):
        assert call(**bad) == EINVAL, bad
    assert call(rows=1 << 31) == EUNSUPPORTED and call(rows=0) == OK

    names = "rows cols type x ldx g b eps y ldy mean rstd stream".split()
    call = _caller(lib.ozk_layernorm, names, dict(
        rows=4, cols=4, type=kind, x=FAKE, ldx=4, g=FAKE, b=FAKE, eps=1e-5, y=FAKE, ldy=4,
        mean=FAKE, rstd=FAKE, stream=None))
    for bad in (dict(type=4), dict(rows=-1), dict(cols=0), dict(ldx=3), dict(ldy=3),
                dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(y=None), dict(y=ODD),
                dict(mean=ctypes.c_void_p(0x1002)), dict(rstd=ODD)):
        assert call(**bad) == EINVAL, bad
    assert call(cols=1 << 31, ldx=1 << 31, ldy=1 << 31) == EUNSUPPORTED and call(rows=0) == OK

    names = "rows cols type dy lddy x ldx g mean rstd dx lddx dg db ws wsb stream".split()
    call = _caller(lib.ozk_layernorm_backward, names, dict(
        rows=4, cols=4, type=kind, dy=FAKE, lddy=4, x=FAKE, ldx=4, g=FAKE, mean=FAKE, rstd=FAKE,
        dx=FAKE, lddx=4, dg=FAKE, db=FAKE, ws=FAKE, wsb=1 << 20, stream=None))
    for bad in (dict(type=4), dict(rows=-1), dict(cols=0), dict(ldx=3), dict(lddy=3),
                dict(lddx=3), dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None),
                dict(dx=ODD), dict(dg=ODD), dict(db=ODD), dict(ws=ODD)):
        assert call(**bad) == EINVAL, bad
    assert call(ws=None, wsb=0) == EWORKSPACE and call(wsb=16) == EWORKSPACE
    assert call(dx=None, dg=None, db=None, ws=None, wsb=0) == OK
    assert call(rows=0, dg=None, db=None, ws=None, wsb=0) == OK
    out = ctypes.c_size_t()
    assert lib.ozk_layernorm_backward_workspace_size(4, 4, 4, ctypes.byref(out)) == EINVAL
    assert lib.ozk_layernorm_backward_workspace_size(4, 4, kind, None) == EINVAL


def test_binding_refuses_host_tensors_and_names():
    a = torch.zeros(4, 4, dtype=torch.float64)
    q = torch.zeros(4, 4, dtype=torch.int8)
    s = torch.zeros(4)
    with pytest.raises(TypeError):
        ozk.ozk_dgemm_epilogue(a, a, 14)
    with pytest.raises(TypeError):
        ozk.ozk_dgemm_epilogue_grad(a, a, a, 14)
    with pytest.raises(TypeError):
        ozk.ozk_int8linear(q, s, q, s)
    with pytest.raises(TypeError):
        ozk.ozk_int8linear(q, s, q, s, dtype=torch.int32)
    for f in (ozk.ozk_int8quant_rows, ozk.ozk_layernorm):
        with pytest.raises(TypeError):
            f(a)
        with pytest.raises(TypeError):
            f(None)
        with pytest.raises(TypeError):
            f(q)
    with pytest.raises(TypeError):
        ozk.ozk_layernorm_backward(a, a, None, a[0], a[0])
    with pytest.raises(ValueError):
        ozk._act("swish")
