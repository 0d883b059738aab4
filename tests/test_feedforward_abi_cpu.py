"""Refusals of the feed-forward operators that need no GPU: the C entry points check their
arguments before any HIP call, the binding checks tensors before it calls them."""
import ctypes
import os
import random

import pytest
import torch

import fp64_gemm_emulation_ozk_amd as ozk

import mx_plan

OK, EINVAL, EWORKSPACE, ERANGE, EUNSUPPORTED = 0, -1, -2, -3, -5
FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: every call below fails validation
ODD = ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ozk.LIB_PATH):
        from fp64_gemm_emulation_ozk_amd.build import build_library
        build_library(verbose=False)
    return ozk.library()


def _caller(f, names, defaults):
    names = names.split()

    def call(**kw):
        assert set(kw) <= set(names)
        args = dict(defaults, **kw)
        return f(*[args[n] for n in names])
    return call


def test_dgemm_gated_refusals(lib):
    call = _caller(lib.ozk_dgemm_gated,
                   "m n k A lda B ldb bias act Z ldz C ldc r scaling ws wsb stream", dict(
                       m=4, n=4, k=4, A=FAKE, lda=4, B=FAKE, ldb=8, bias=FAKE, act=4, Z=FAKE,
                       ldz=8, C=FAKE, ldc=4, r=14, scaling=0, ws=FAKE, wsb=1 << 20, stream=None))
    for bad in (dict(act=-1), dict(act=5), dict(r=0), dict(r=21), dict(scaling=2), dict(m=-1),
                dict(n=-1), dict(k=0), dict(lda=3), dict(ldb=7), dict(ldc=3), dict(ldz=7),
                dict(A=None), dict(B=None), dict(C=None), dict(ws=ODD)):
        assert call(**bad) == EINVAL, bad
    assert call(k=131072, lda=131072) == ERANGE
    assert call(r=2, k=1 << 16, lda=1 << 16) == ERANGE          # no bit budget
    assert call(n=1 << 41, ldb=1 << 42, ldc=1 << 41) == EUNSUPPORTED
    assert call(ws=None, wsb=0) == EWORKSPACE and call(wsb=16) == EWORKSPACE
    assert call(m=0, ws=None, wsb=0) == OK and call(n=0, ws=None, wsb=0) == OK
    out = ctypes.c_size_t()
    size = lib.ozk_dgemm_gated_workspace_size
    assert size(4, 4, 4, 14, None) == EINVAL and size(4, 4, 0, 14, ctypes.byref(out)) == EINVAL
    assert size(4, 4, 131072, 14, ctypes.byref(out)) == ERANGE
    for n in (1, 31, 33, 64, 100):
        assert size(4, n, 4, 14, ctypes.byref(out)) == OK
        # a row of residues holds whole groups of 64 from column 0 and from column n on
        assert out.value >= 14 * 4 * (n + (n + 63) // 64 * 64)
        assert call(n=n, ldb=2 * n, ldc=n, ldz=2 * n, wsb=out.value - 1) == EWORKSPACE
    assert call(Z=None, ldz=0, wsb=16) == EWORKSPACE   # an absent Z asks nothing of ldz


def test_dgemm_gated_grad_refusals(lib):
    call = _caller(lib.ozk_dgemm_gated_grad, "m n k dC lddc A lda B ldb Z ldz act dA ldda dB lddb "
                   "db r scaling ws wsb stream", dict(
                       m=4, n=4, k=4, dC=FAKE, lddc=4, A=FAKE, lda=4, B=FAKE, ldb=8, Z=FAKE, ldz=8,
                       act=0, dA=FAKE, ldda=4, dB=FAKE, lddb=8, db=FAKE, r=14, scaling=1, ws=FAKE,
                       wsb=1 << 30, stream=None))
    for bad in (dict(act=5), dict(r=0), dict(scaling=-1), dict(n=-1), dict(m=-1), dict(k=0),
                dict(lddc=3), dict(ldz=7), dict(ldda=3), dict(lddb=7), dict(lda=3), dict(ldb=7),
                dict(dC=None), dict(Z=None), dict(A=None), dict(B=None), dict(ws=ODD)):
        assert call(**bad) == EINVAL, bad
    assert call(m=131072) == ERANGE and call(n=65536) == ERANGE and call(k=131072) == ERANGE
    assert call(r=2, m=1 << 16, scaling=0) == ERANGE            # dB's budget
    assert call(ws=None, wsb=0) == EWORKSPACE and call(wsb=256) == EWORKSPACE
    assert call(dA=None, dB=None, db=None, ws=None, wsb=0) == OK
    assert call(m=0, dB=None, db=None, ws=None, wsb=0) == OK    # dA has no rows
    out = ctypes.c_size_t()
    size = lib.ozk_dgemm_gated_grad_workspace_size
    assert size(4, 4, 4, 14, None) == EINVAL and size(4, 65536, 4, 14, None) == EINVAL
    assert size(4, 65536, 4, 14, ctypes.byref(out)) == ERANGE
    assert size(4, 65536, 4, 0, ctypes.byref(out)) == EINVAL
    assert size(64, 48, 32, 14, ctypes.byref(out)) == OK
    assert out.value >= 8 * 64 * 96 + 14 * (64 + 32) * 128 + 14 * 64 * 32


def test_mxfp4_sizes(lib):
    for k, steps in ((1, 1), (255, 1), (256, 1), (257, 2), (131071, 512)):
        assert lib.ozk_mxfp4_line_bytes(k) == ozk.ozk_mxfp4_line_bytes(k) == 128 * steps
        assert lib.ozk_mxfp4_scale_bytes(k) == ozk.ozk_mxfp4_scale_bytes(k) == 8 * steps
    assert lib.ozk_mxfp4_line_bytes(0) == 0 and lib.ozk_mxfp4_scale_bytes(-1) == 0


@pytest.mark.parametrize("kind", [0, 1, 2, 3])
def test_mxfp4_codes_refusals(lib, kind):
    call = _caller(lib.ozk_mxfp4_quant, "rows cols type x ldx axis q ldq s lds stream", dict(
        rows=4, cols=4, type=kind, x=FAKE, ldx=4, axis=0, q=FAKE, ldq=128, s=FAKE, lds=8,
        stream=None))
    for bad in (dict(type=4), dict(type=-1), dict(axis=2), dict(axis=-1), dict(rows=-1),
                dict(cols=0), dict(cols=-1), dict(axis=1, rows=0), dict(ldx=3), dict(x=None),
                dict(q=None), dict(s=None), dict(x=ODD), dict(q=ctypes.c_void_p(0x1008)),
                dict(s=ctypes.c_void_p(0x1004)), dict(ldq=136), dict(ldq=112), dict(lds=12),
                dict(lds=0), dict(cols=257, ldx=257), dict(axis=1, rows=257),
                dict(cols=257, ldx=257, ldq=256)):
        assert call(**bad) == EINVAL, bad
    assert call(rows=0) == OK and call(axis=1, cols=0) == OK
    assert call(rows=1 << 31) == EUNSUPPORTED and call(cols=1 << 31, ldx=1 << 31) == EUNSUPPORTED

    call = _caller(lib.ozk_mxfp4_values, "lines k q ldq s lds type out ldo stream", dict(
        lines=4, k=4, q=FAKE, ldq=128, s=FAKE, lds=8, type=kind, out=FAKE, ldo=4, stream=None))
    for bad in (dict(type=4), dict(type=-1), dict(lines=-1), dict(k=0), dict(ldo=3),
                dict(q=None), dict(s=None), dict(out=None), dict(out=ODD), dict(q=ODD),
                dict(s=ODD), dict(ldq=120), dict(lds=4), dict(k=300, ldo=300)):
        assert call(**bad) == EINVAL, bad
    assert call(lines=0) == OK
    assert call(lines=1 << 31) == EUNSUPPORTED and call(k=1 << 31, ldo=1 << 31) == EUNSUPPORTED


@pytest.mark.parametrize("gated", [False, True])
def test_mxfp4_product_refusals(lib, gated):
    f = lib.ozk_mxfp4_gated if gated else lib.ozk_mxfp4_linear
    size = lib.ozk_mxfp4_gated_workspace_size if gated else lib.ozk_mxfp4_linear_workspace_size
    names = ("m n k X ldx sx ldsx W ldw sw ldsw bias act " + ("" if gated else "R ldr ")
             + "type C ldc ws wsb stream")
    defaults = dict(m=4, n=4, k=4, X=FAKE, ldx=128, sx=FAKE, ldsx=8, W=FAKE, ldw=128, sw=FAKE,
                    ldsw=8, bias=FAKE, act=0, type=3, C=FAKE, ldc=4, ws=None, wsb=0, stream=None)
    if not gated:
        defaults.update(R=FAKE, ldr=4)
    call = _caller(f, names, defaults)
    bads = [dict(act=5), dict(act=-1), dict(type=0), dict(type=4), dict(type=-1), dict(m=-1),
            dict(n=-1), dict(k=0), dict(k=257), dict(ldx=120), dict(ldw=0), dict(ldsx=4),
            dict(ldsw=12), dict(ldc=3), dict(X=None), dict(W=None), dict(sx=None), dict(sw=None),
            dict(C=None), dict(X=ctypes.c_void_p(0x1008)), dict(W=ODD), dict(sw=ODD),
            dict(sx=ctypes.c_void_p(0x1004)), dict(bias=ODD), dict(C=ODD)]
    if not gated:
        bads += [dict(ldr=3), dict(R=ODD)]
    for bad in bads:
        assert call(**bad) == EINVAL, bad
    assert call(k=131073, ldx=1 << 17, ldw=1 << 17, ldsx=1 << 13, ldsw=1 << 13) == ERANGE
    assert call(m=1 << 31) == EUNSUPPORTED and call(n=1 << 30, ldc=1 << 30, **(
        {} if gated else dict(ldr=1 << 30))) == EUNSUPPORTED
    for ld in ("ldx", "ldw", "ldsx", "ldsw"):
        assert call(**{ld: 1 << 24}) == EUNSUPPORTED
    assert call(m=0) == OK and call(n=0) == OK
    out = ctypes.c_size_t()
    assert size(4, 4, 0, ctypes.byref(out)) == EINVAL and size(4, 4, 4, None) == EINVAL
    assert size(4, -1, 4, ctypes.byref(out)) == EINVAL
    assert size(4, 4, 131073, ctypes.byref(out)) == ERANGE
    assert size(4, 4, 131072, ctypes.byref(out)) == OK
    assert size(0, 4, 4, ctypes.byref(out)) == OK and out.value == 0
    # a launch that would pass 2^32 threads
    big = dict(m=1 << 22, n=1 << 22, ldc=1 << 22, ws=FAKE, wsb=1 << 62)
    assert call(**big, **({} if gated else dict(ldr=1 << 22))) == EUNSUPPORTED
    # where a workspace is needed it is asked for
    for m, n, k in ((1, 16, 131071), (40, 200, 65536), (100, 100, 16384)):
        assert size(m, n, k, ctypes.byref(out)) == OK
        lb, sb = ozk.ozk_mxfp4_line_bytes(k), ozk.ozk_mxfp4_scale_bytes(k)
        args = dict(m=m, n=n, k=k, ldx=lb, ldw=lb, ldsx=sb, ldsw=sb, ldc=n)
        if not gated:
            args["ldr"] = n
        if out.value:
            assert call(**args) == EWORKSPACE and call(**args, ws=FAKE) == EWORKSPACE
            assert call(**args, ws=FAKE, wsb=out.value - 1) == EWORKSPACE
            assert call(**args, ws=ODD, wsb=out.value) == EINVAL


def test_the_plan_of_the_tests_is_the_library_s(lib):
    """How often K is split shows in the workspace, over sizes spread over the whole range."""
    rng = random.Random(5)
    out = ctypes.c_size_t()
    sizes = mx_plan.TILES + mx_plan.STREAM + [
        [int(2 ** rng.uniform(0, top)) for top in (13, 14, 17)] for _ in range(4000)]
    split = 0
    for m, n, k in sizes:
        for gated, f in ((False, lib.ozk_mxfp4_linear_workspace_size),
                         (True, lib.ozk_mxfp4_gated_workspace_size)):
            assert f(m, n, k, ctypes.byref(out)) == OK
            splits = mx_plan.plan(m, n, k, gated)[1]
            split += splits > 1
            need = splits * m * n * (8 if gated else 4) if splits > 1 else 0
            assert out.value == (need + 255) // 256 * 256, (m, n, k, gated, splits)
    assert split > 1000


@pytest.mark.parametrize("gated", [False, True])
def test_sizes_take_every_kernel_into_its_steady_state(gated):
    """Each tile, K whole and split, over more steps than twice what its rings of codes and of
    scales hold, in odd and even numbers; each width of the streams over more steps a wave than
    any ring of theirs (three)."""
    tiles, streams = {}, {}
    for m, n, k in mx_plan.TILES:
        shape, splits = mx_plan.plan(m, n, k, gated)
        steps = mx_plan.steps_of(k)
        firsts = [steps * s // splits for s in range(splits + 1)]
        tiles.setdefault((shape, splits > 1), []).extend(
            (firsts[s] % 2, firsts[s + 1] - firsts[s]) for s in range(splits))
    assert set(tiles) == {(s, split) for s in ("small", "mid", "large") for split in (False, True)}
    for (shape, split), runs in tiles.items():
        around = 2 * max(4 * mx_plan.SCALE_BUFFERS[shape], mx_plan.CODE_STAGES[shape])
        assert any(count > around for _, count in runs), (shape, split)
        assert not split or {odd for odd, _ in runs} == {0, 1}
    for shape in ("mid", "large"):
        assert {5, 8, 9, 13, 17} <= {count for _, count in tiles[shape, False]}
    for m, n, k in mx_plan.STREAM:
        kernel, splits = mx_plan.plan(m, n, k, gated)
        streams.setdefault(kernel, []).append(-(-(mx_plan.steps_of(k) // splits) // 8))
    assert set(streams) == {("stream", r, c) for r in (8, 16, 32, 64) for c in (1, 2)}
    for waves in streams.values():
        assert 1 in waves and max(waves) > 3


def _clip(lib, tensors, max_norm=1.0, norm=FAKE, ws=FAKE, wsb=1 << 20):
    """tensors: (x, out, size, type)"""
    n = len(tensors)
    xs = (ctypes.c_void_p * n)(*[t[0] for t in tensors])
    ys = (ctypes.c_void_p * n)(*[t[1] for t in tensors])
    sizes = (ctypes.c_int64 * n)(*[t[2] for t in tensors])
    types = (ctypes.c_int * n)(*[t[3] for t in tensors])
    return lib.ozk_clip_norm(n, xs, ys, sizes, types, max_norm, norm, ws, wsb, None)


def test_clip_norm_refusals(lib):
    a, b = 0x10000, 0x20000
    good = (a, b, 16, 1)
    for bad in ([(None, b, 16, 1)], [(a, None, 16, 1)], [(a, b, -1, 1)], [(a, b, 16, 4)],
                [(a, b, 16, -1)], [(a + 1, b, 16, 1)], [(a, b + 2, 16, 1)], [(a, b + 4, 16, 0)],
                [(a, a + 4, 16, 1)],                      # an output over its own input, shifted
                [(a, b, 16, 1), (a, b, 16, 1)],           # one output twice
                [(a, a, 16, 1), (a, a, 16, 1)],           # one tensor twice, in place
                [(a, b, 16, 1), (a + 64, b + 60, 16, 1)],
                [(a, b, 16, 1), (b, a + 4096, 16, 1)],    # an output is another's input
                [(a, b, 16, 1)] * 65 + [(a, b, 16, 1)]):
        assert _clip(lib, bad) == EINVAL, bad
    for kw in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(norm=None),
               dict(norm=ctypes.c_void_p(0x1004)), dict(ws=ODD)):
        assert _clip(lib, [good], **kw) == EINVAL, kw
    for at in (a, a + 56, b, b + 56):                          # the norm among the values
        assert _clip(lib, [good], norm=ctypes.c_void_p(at)) == EINVAL, at
    assert _clip(lib, [good], wsb=16) == EWORKSPACE and _clip(lib, [good], ws=None) == EWORKSPACE
    assert _clip(lib, [(a, b, 1 << 43, 1)]) == EUNSUPPORTED
    f = lib.ozk_clip_norm
    assert f(-1, None, None, None, None, 1.0, FAKE, FAKE, 1 << 20, None) == EINVAL
    assert f(1, None, None, None, None, 1.0, FAKE, FAKE, 1 << 20, None) == EINVAL
    out = ctypes.c_size_t()
    size = lib.ozk_clip_norm_workspace_size
    assert size(-1, ctypes.byref(out)) == EINVAL and size(4, None) == EINVAL
    assert size(1 << 23, ctypes.byref(out)) == EUNSUPPORTED
    assert size(0, ctypes.byref(out)) == OK and out.value == 0
    assert size(1, ctypes.byref(out)) == OK and _clip(lib, [good], wsb=out.value - 1) == EWORKSPACE
    # the overlap check passes tensors side by side (what is refused here is the workspace)
    assert _clip(lib, [(a, b, 16, 1), (a, b + 64, 16, 1), (a + 64, a + 64, 16, 1)],
                 ws=None) == EWORKSPACE


def test_limits_are_where_they_are_stated(lib):
    """The first value that is refused as unsupported, and the last that is not: with no
    workspace the latter are refused for that.  No call gets past the checks."""
    call = _caller(lib.ozk_dgemm_gated,
                   "m n k A lda B ldb bias act Z ldz C ldc r scaling ws wsb stream", dict(
                       m=1, n=4, k=4, A=FAKE, lda=4, B=FAKE, ldb=1 << 42, bias=None, act=4, Z=None,
                       ldz=0, C=FAKE, ldc=1 << 42, r=14, scaling=0, ws=None, wsb=0, stream=None))
    out = ctypes.c_size_t()
    size = lib.ozk_dgemm_gated_workspace_size
    for n, unsupported in ((1 << 40, True), ((1 << 40) - 1, False)):
        assert call(n=n) == (EUNSUPPORTED if unsupported else EWORKSPACE)
        assert size(1, n, 4, 14, ctypes.byref(out)) == (EUNSUPPORTED if unsupported else OK)

    a = 1 << 50
    for kind, e in ((0, 8), (1, 4), (2, 2), (3, 2)):
        most = (1 << 44) // e
        assert _clip(lib, [(a, a, most, kind)], ws=None) == EUNSUPPORTED
        assert _clip(lib, [(a, a, most - 1, kind)], ws=None) == EWORKSPACE
    # of all: 2^45 bytes with 2^15 for each tensor
    for last, status in (((1 << 43) - 3 * 32768, EUNSUPPORTED),
                         ((1 << 43) - 3 * 32768 - 8, EWORKSPACE)):
        each = [1 << 43, 1 << 43, 1 << 43, last - 32768]
        tensors = [(a + (i << 44), a + (i << 44), b // 8, 0) for i, b in enumerate(each)]
        assert _clip(lib, tensors + [(a, a, 0, 0)], ws=None) == status

    for f in (lib.ozk_mxfp4_linear_workspace_size, lib.ozk_mxfp4_gated_workspace_size):
        for m, n, status in (((1 << 31) - 1, 1, OK), (1 << 31, 1, EUNSUPPORTED),
                             (1, (1 << 30) - 1, OK), (1, 1 << 30, EUNSUPPORTED)):
            assert f(m, n, 256, ctypes.byref(out)) == status
    size = lib.ozk_clip_norm_workspace_size
    assert size((1 << 23) - 1, ctypes.byref(out)) == OK


def test_binding_refuses_host_tensors_and_names():
    a = torch.zeros(4, 4, dtype=torch.float64)
    q = torch.zeros(4, 128, dtype=torch.uint8)
    s = torch.zeros(4, 8, dtype=torch.uint8)
    with pytest.raises(TypeError):
        ozk.ozk_dgemm_gated(a, a, 14)
    with pytest.raises(TypeError):
        ozk.ozk_dgemm_gated_grad(a, a, a, 14, a)
    for f in (ozk.ozk_mxfp4_linear, ozk.ozk_mxfp4_gated):
        with pytest.raises(TypeError):
            f(q, s, q, s)
        for dtype in (torch.float64, torch.int32):
            with pytest.raises(TypeError):
                f(q, s, q, s, dtype=dtype)
    with pytest.raises(TypeError):
        ozk.ozk_mxfp4_values(q, s)
    for bad in (a, None, q):
        with pytest.raises(TypeError):
            ozk.ozk_mxfp4_quant(bad)
    with pytest.raises(TypeError):
        ozk.ozk_clip_norm([a], 1.0)
    with pytest.raises(TypeError):
        ozk.ozk_clip_norm([None], 1.0)
    with pytest.raises(ValueError):
        ozk.ozk_clip_norm([], 1.0)
    with pytest.raises(ValueError):
        ozk.ozk_clip_norm([a, a], 1.0, out=[a])
