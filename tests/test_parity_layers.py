"""GPU parity of the layer operators against their plain 64-bit forms.

Tolerances count roundings.  u = 2^-24 (2^-53) is half a step of the fp32 (fp64) arithmetic,
eps / 2 of the output's type one rounding to it.  A sum of terms t_i taken in D steps is off
by at most D u sum |t_i|."""
import numpy as np
import pytest
import torch

import fp64_gemm_emulation_ozk_amd as ozk
import ozk_inputs
from oracle import layers, ozaki2

from gpu_common import announce, device, to_dev

pytestmark = pytest.mark.gpu

TYPES = {"float64": torch.float64, "float32": torch.float32, "float16": torch.float16,
         "bfloat16": torch.bfloat16}
U32, U64 = 2.0 ** -24, 2.0 ** -53


def host(t):
    return t.detach().double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the spacing of dtype's subnormals (float64: zero is exact enough)."""
    fi = torch.finfo(dtype)
    return fi.tiny * fi.eps / 2


def assert_near(got, want, tol, what):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    if bad.any():
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, worst "
                             f"{np.nanmax(err / np.maximum(tol, 1e-300)):.3g} of the tolerance "
                             f"at {np.argwhere(bad)[0].tolist()}")


def padded(x, pad, offset=0):
    """x on the device as a view of a wider buffer: leading dimension cols + pad, its first
    element `offset` elements past an aligned one."""
    rows, cols = x.shape
    buf = torch.empty(offset + rows * (cols + pad), dtype=x.dtype, device=device())
    v = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(x.to(device()))
    return v


# ------------------------------------------------------------------ rows
# columns: below, at and above a vector; each registers-per-thread shape and the first length
# past it for 8, 4 and 2 elements a vector; a row beyond registers
COLS = [1, 2, 3, 7, 64, 65, 130, 513, 1000, 1024, 1537, 2049, 4096, 4100, 8193, 16384, 20001,
        32769, 40000]


def rows_of(cols):
    return 5 if cols > 3000 else 13


def row_input(rows, cols, dtype, seed, mean=0.3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, dtype=torch.float64)
    x = x * torch.exp(torch.randn(rows, 1, generator=g, dtype=torch.float64)) + mean
    gamma = (1 + 0.3 * torch.randn(cols, generator=g, dtype=torch.float64)).to(dtype)
    beta = (0.3 * torch.randn(cols, generator=g, dtype=torch.float64)).to(dtype)
    dy = torch.randn(rows, cols, generator=g, dtype=torch.float64).to(dtype)
    return x.to(dtype), gamma, beta, dy


def depth(cols):
    """Additions a term passes in a row's sum: at most 32 in a thread that holds the row in
    registers, cols / 1024 in one that walks it, and 32 across threads (6 in a wave, 16
    between waves)."""
    return max(32, cols // 1024 + 8) + 32


def norm_bounds(x, gamma, beta, eps, u, cols):
    """(y, mean, rstd) in 64 bits and bounds of what arithmetic with unit u may be off."""
    y, mean, rstd = layers.layernorm(x, gamma, beta, eps)
    d = depth(cols)
    e_mean = (d + 2) * u * np.abs(x).mean(1)
    dev = x - mean[:, None]
    e_dev = e_mean[:, None] + u * (np.abs(dev) + e_mean[:, None])
    var = (dev ** 2).mean(1)
    # mean of (dev + e)^2: the first-order part sums e_mean * dev, which is e_mean times
    # sum(dev) = 0 up to the roundings, so 2 u |dev| |dev| and e^2 remain; taken whole here
    e_var = (2 * np.abs(dev) * e_dev + e_dev ** 2).mean(1) + (d + 4) * u * var
    r_rel = np.minimum(0.5 * e_var / (var + eps) * 1.5 + 4 * u, 1.0)
    e_rstd = rstd * r_rel
    g = np.ones(cols) if gamma is None else gamma
    e_y = (np.abs(g) * rstd[:, None] * (e_dev + np.abs(dev) * r_rel[:, None]) * 1.01
           + 4 * u * (np.abs(dev * rstd[:, None] * g) + np.abs(y)))
    return (y, mean, rstd), (e_y, e_mean, e_rstd)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("cols", COLS)
def test_layernorm(kind, cols):
    announce(f"layernorm {kind} cols={cols}")
    dtype, rows = TYPES[kind], rows_of(cols)
    u = U64 if kind == "float64" else U32
    x, gamma, beta, _ = row_input(rows, cols, dtype, cols)
    for weights in (True, False):
        gm, bt = (gamma, beta) if weights else (None, None)
        for pad, offset in ((0, 0), (3, 1)):
            xd = padded(x, pad, offset)
            out = padded(torch.full((rows, cols), 7.0, dtype=dtype), pad + 1, offset)
            y, mean, rstd = ozk.ozk_layernorm(
                xd, gm.to(device()) if weights else None, bt.to(device()) if weights else None,
                eps=1e-5, stats=True, out=out)
            assert y is out
            (wy, wm, wr), (ey, em, er) = norm_bounds(
                host(x), host(gm) if weights else None, host(bt) if weights else None, 1e-5, u,
                cols)
            assert_near(host(y), wy, ey + half_step(dtype) * (np.abs(wy) + ey) + tiny(dtype),
                        "y")
            assert_near(host(mean), wm, em + 1e-300, "mean")
            assert_near(host(rstd), wr, er + u * wr, "rstd")


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("cols", COLS)
def test_layernorm_backward(kind, cols):
    announce(f"layernorm backward {kind} cols={cols}")
    dtype, rows = TYPES[kind], rows_of(cols)
    u = U64 if kind == "float64" else U32
    stat = torch.float64 if kind == "float64" else torch.float32
    x, gamma, _, dy = row_input(rows, cols, dtype, cols + 1)
    _, m, r = layers.layernorm(host(x))
    mean, rstd = torch.from_numpy(m).to(stat), torch.from_numpy(r).to(stat)
    for weights, pad in ((True, 0), (True, 5), (False, 1)):
        gm = gamma if weights else None
        dx, dg, db = ozk.ozk_layernorm_backward(
            padded(dy, pad), padded(x, 2 * pad, pad), gm.to(device()) if weights else None,
            mean.to(device()), rstd.to(device()))
        hx, hdy, hm, hr = host(x), host(dy), host(mean), host(rstd)
        hg = host(gm) if weights else np.ones(cols)
        want = layers.layernorm_backward(hdy, hx, hg, hm, hr)
        xh = (hx - hm[:, None]) * hr[:, None]
        g = hdy * hg
        n = cols
        c1, c2 = (g * xh).mean(1), g.mean(1)
        e1 = (depth(cols) + 6) * u * np.abs(g * xh).mean(1)
        e2 = (depth(cols) + 4) * u * np.abs(g).mean(1)
        ex = hr[:, None] * (e2[:, None] + np.abs(xh) * e1[:, None]
                            + 6 * u * (np.abs(g) + np.abs(c2)[:, None]
                                       + np.abs(xh * c1[:, None]))) * 1.01
        assert_near(host(dx), want[0], ex + half_step(dtype) * (np.abs(want[0]) + ex)
                    + tiny(dtype), "dx")
        # at most rows + 32 additions a column (16 slices of row groups, then the slices)
        eg = (rows + 36) * u * np.abs(hdy * xh).sum(0)
        eb = (rows + 34) * u * np.abs(hdy).sum(0)
        assert_near(host(dg), want[1], eg + half_step(dtype) * (np.abs(want[1]) + eg)
                    + tiny(dtype), "dgamma")
        assert_near(host(db), want[2], eb + half_step(dtype) * (np.abs(want[2]) + eb)
                    + tiny(dtype), "dbeta")


@pytest.mark.parametrize("rows,cols", [(1, 64), (511, 65), (513, 300), (3000, 130), (1100, 2100)])
def test_layernorm_backward_many_rows(rows, cols):
    """More rows than row groups, and the sums joined the same way every time."""
    announce(f"layernorm backward rows={rows} cols={cols}")
    x, gamma, _, dy = row_input(rows, cols, torch.float32, rows)
    _, m, r = layers.layernorm(host(x))
    args = [t.to(device()) for t in (dy, x, gamma, torch.from_numpy(m).float(),
                                     torch.from_numpy(r).float())]
    first = ozk.ozk_layernorm_backward(*args)
    again = ozk.ozk_layernorm_backward(*args)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    hm, hr = host(args[3]), host(args[4])
    want = layers.layernorm_backward(host(dy), host(x), host(gamma), hm, hr)
    xh = (host(x) - hm[:, None]) * hr[:, None]
    d = rows // 64 + 64   # rows of a group in order, groups of a slice, slices
    assert_near(host(first[1]), want[1], (d + 4) * U32 * np.abs(host(dy) * xh).sum(0), "dgamma")
    assert_near(host(first[2]), want[2], (d + 2) * U32 * np.abs(host(dy)).sum(0), "dbeta")


# every shape of workgroup with more rows than it has at once: 64, 256 and 1024 threads, one and
# two vectors each, gamma kept in registers and read again for each row
@pytest.mark.parametrize("kind,rows,cols", [
    ("float32", 2600, 130), ("float32", 2500, 400), ("float32", 1100, 1000),
    ("float32", 1100, 2048), ("float32", 600, 4000), ("float32", 600, 7001),
    ("bfloat16", 2200, 300), ("bfloat16", 1030, 4096), ("bfloat16", 600, 16384),
    ("float16", 600, 8200), ("float64", 2100, 65), ("float64", 600, 2000), ("float64", 520, 4096)])
def test_layernorm_backward_rows_in_turn(kind, rows, cols):
    """Rows that a workgroup takes one after the other: dx of every row, also over dy and x while
    the next row is on its way."""
    announce(f"layernorm backward rows in turn {kind} rows={rows} cols={cols}")
    dtype = TYPES[kind]
    u = U64 if kind == "float64" else U32
    stat = torch.float64 if kind == "float64" else torch.float32
    x, gamma, _, dy = row_input(rows, cols, dtype, rows + cols)
    _, m, r = layers.layernorm(host(x))
    dyd, xd, gd, md, rd = [t.to(device()) for t in (dy, x, gamma, torch.from_numpy(m).to(stat),
                                                    torch.from_numpy(r).to(stat))]
    got = ozk.ozk_layernorm_backward(dyd, xd, gd, md, rd)
    hx, hdy, hg, hm, hr = host(x), host(dy), host(gamma), host(md), host(rd)
    want = layers.layernorm_backward(hdy, hx, hg, hm, hr)
    xh = (hx - hm[:, None]) * hr[:, None]
    g = hdy * hg
    c1, c2 = (g * xh).mean(1), g.mean(1)
    # as in test_layernorm_backward
    e1 = (depth(cols) + 6) * u * np.abs(g * xh).mean(1)
    e2 = (depth(cols) + 4) * u * np.abs(g).mean(1)
    ex = hr[:, None] * (e2[:, None] + np.abs(xh) * e1[:, None]
                        + 6 * u * (np.abs(g) + np.abs(c2)[:, None]
                                   + np.abs(xh * c1[:, None]))) * 1.01
    assert_near(host(got[0]), want[0], ex + half_step(dtype) * (np.abs(want[0]) + ex)
                + tiny(dtype), "dx")
    d = rows // 64 + 64   # rows of a group in order, groups of a slice, slices
    for out, w, t, what in ((got[1], want[1], hdy * xh, "dgamma"), (got[2], want[2], hdy, "dbeta")):
        e = (d + 4) * u * np.abs(t).sum(0)
        assert_near(host(out), w, e + half_step(dtype) * (np.abs(w) + e) + tiny(dtype), what)
    for which in (0, 1):
        a, b = dyd.clone(), xd.clone()
        over = ozk.ozk_layernorm_backward(a, b, gd, md, rd, dx=(a, b)[which])
        for o, w in zip(over, got):
            assert torch.equal(o, w)


def test_layernorm_backward_parts():
    """dx alone needs no workspace; dgamma and dbeta alone leave dx; in place over dy and x;
    no rows give zero sums."""
    announce("layernorm backward parts")
    x, gamma, _, dy = row_input(9, 200, torch.float32, 3)
    _, m, r = layers.layernorm(host(x))
    dy, x, gamma, m, r = [t.to(device()) for t in (dy, x, gamma, torch.from_numpy(m).float(),
                                                   torch.from_numpy(r).float())]
    dx, dg, db = ozk.ozk_layernorm_backward(dy, x, gamma, m, r)
    only, none1, none2 = ozk.ozk_layernorm_backward(dy, x, gamma, m, r, need_weights=False)
    assert none1 is None and none2 is None and torch.equal(only, dx)
    none, g2, b2 = ozk.ozk_layernorm_backward(dy, x, gamma, m, r, need_dx=False)
    assert none is None and torch.equal(g2, dg) and torch.equal(b2, db)
    for which in (0, 1):
        a, b = dy.clone(), x.clone()
        got = ozk.ozk_layernorm_backward(a, b, gamma, m, r, dx=(a, b)[which])
        assert torch.equal(got[0], dx) and torch.equal(got[1], dg)
    e = torch.empty((0, 200), device=device())
    z = torch.empty(0, device=device())
    dx0, dg0, db0 = ozk.ozk_layernorm_backward(e, e, gamma, z, z)
    assert dx0.shape == (0, 200) and not dg0.any() and not db0.any()


@pytest.mark.parametrize("kind,cols", [("float32", 700), ("bfloat16", 16400), ("float32", 40000)])
def test_layernorm_in_place(kind, cols):
    """The output over an input, also where a row does not fit registers (the gradient's column
    sums then read dy and x in a launch of their own)."""
    announce(f"layernorm in place {kind} cols={cols}")
    dtype = TYPES[kind]
    x, gamma, beta, dy = [t.to(device()) for t in row_input(21, cols, dtype, cols + 9)]
    y, mean, rstd = ozk.ozk_layernorm(x, gamma, beta, stats=True)
    over = x.clone()
    assert torch.equal(ozk.ozk_layernorm(over, gamma, beta, out=over), y)
    want = ozk.ozk_layernorm_backward(dy, x, gamma, mean, rstd)
    for which in (0, 1):
        a, b = dy.clone(), x.clone()
        got = ozk.ozk_layernorm_backward(a, b, gamma, mean, rstd, dx=(a, b)[which])
        for g, w in zip(got, want):
            assert torch.equal(g, w)


def test_rows_of_several_launches():
    """More rows than one launch takes: the same bits as those rows alone."""
    announce("rows of several launches")
    block, gamma, beta, _ = row_input(1027, 8, torch.float16, 11)
    rows = (1 << 21) + 1030
    x = block.to(device()).repeat(rows // 1027 + 1, 1)[:rows].contiguous()
    gm, bt = gamma.to(device()), beta.to(device())
    y, mean, rstd = ozk.ozk_layernorm(x, gm, bt, stats=True)
    q, scale = ozk.ozk_int8quant_rows(x, norm=True, gamma=gm, beta=bt)
    alone = ozk.ozk_layernorm(x[:1027], gm, bt, stats=True)
    codes = ozk.ozk_int8quant_rows(x[:1027], norm=True, gamma=gm, beta=bt)
    for got, want in zip((y, mean, rstd, q, scale), alone + codes):
        want = want.repeat((rows // 1027 + 1,) + (1,) * (want.dim() - 1))[:rows]
        assert torch.equal(got, want)


def test_layernorm_backward_columns_of_several_launches():
    """2^27 columns and some: their sums are joined by more than one launch.  One row, so each sum
    is one term: dy itself and dy xh, rounded as torch rounds the same fp32 steps."""
    cols = (1 << 27) + 5
    announce(f"layernorm backward cols={cols}")
    g = torch.Generator(device=device()).manual_seed(8)
    dy = torch.randn(1, cols, generator=g, device=device())
    x = torch.randn(1, cols, generator=g, device=device())
    mean, rstd = torch.tensor([0.25], device=device()), torch.tensor([1.5], device=device())
    _, dgamma, dbeta = ozk.ozk_layernorm_backward(dy, x, None, mean, rstd, need_dx=False)
    assert torch.equal(dbeta, dy[0])
    assert torch.equal(dgamma, (dy * ((x - mean) * rstd))[0])


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("cols", [1, 5, 130, 777, 1537, 4096, 5000, 20001, 40000])
def test_layernorm_far_from_zero(kind, cols):
    """Rows of one value: y is zero.  Rows about a far value: the mean of a sum in fp32 is off by
    e = (depth + 2) u |value|, x - mean is exact (Sterbenz), and the sum of those differences,
    each at most |dev| + e, gives the rest of the mean within (depth + 4) u of their mean."""
    announce(f"layernorm far from zero {kind} cols={cols}")
    dtype = TYPES[kind]
    values = (0.1, 3.3, -1000.1, 12345.6)
    d = depth(cols)
    flat = torch.tensor(values).to(dtype)[:, None].repeat(1, cols)
    y, mean, rstd = ozk.ozk_layernorm(flat.to(device()), stats=True)
    # what is left of the mean, (d + 4) u e, over sqrt(eps); the mean is the value itself but for
    # one rounding, the variance e^2 (d + 6) u at most
    e = (d + 2) * U32 * np.abs(host(flat))
    left = (d + 4) * U32 * e / np.sqrt(1e-5)
    assert_near(host(y), np.zeros(flat.shape), left * (1 + half_step(dtype)) + tiny(dtype), "flat")
    assert_near(host(mean), host(flat)[:, 0], U32 * np.abs(host(flat)[:, 0]), "mean")
    if cols < 100:
        return
    g = torch.Generator().manual_seed(cols)
    x = (torch.randn(4, cols, generator=g) + torch.tensor(values)[:, None]).to(dtype)
    y, mean, rstd = ozk.ozk_layernorm(x.to(device()), stats=True)
    wy, wm, wr = layers.layernorm(host(x))
    dev = np.abs(host(x) - wm[:, None])
    e = (d + 2) * U32 * np.abs(host(x)).mean(1)
    each = dev + e[:, None]
    e_dev = (d + 4) * U32 * each.mean(1)[:, None] + 2 * U32 * each
    r_rel = 0.75 * ((2 * dev * e_dev + e_dev ** 2).mean(1) + (d + 6) * U32 * (each ** 2).mean(1)) \
        * wr ** 2 + 4 * U32
    ey = 1.01 * wr[:, None] * (e_dev + dev * r_rel[:, None]) + 4 * U32 * np.abs(wy)
    assert_near(host(y), wy, ey + half_step(dtype) * (np.abs(wy) + ey) + tiny(dtype), "y")
    assert_near(host(mean), wm, e_dev.max(1) + U32 * np.abs(wm), "mean")
    assert_near(host(rstd), wr, wr * (r_rel + U32), "rstd")


def test_layernorm_edges():
    """A large common offset (two passes: no cancellation), a constant row, rows with NaN and
    Inf beside sound ones, in place, no rows."""
    announce("layernorm edges")
    g = torch.Generator().manual_seed(5)
    x = torch.randn(6, 777, generator=g, dtype=torch.float64).float()
    x[0] += 4096.0
    x[1] = 3.25
    x[2, 5], x[3, 7] = float("nan"), float("inf")
    y, mean, rstd = ozk.ozk_layernorm(x.to(device()), stats=True)
    for i in (0, 4, 5):
        (wy, _, _), (ey, _, _) = norm_bounds(host(x[i:i + 1]), None, None, 1e-5, U32, 777)
        assert_near(host(y[i:i + 1]), wy, ey + U32 * np.abs(wy), f"row {i}")
    assert not y[1].any() and float(mean[1]) == 3.25
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    xd = x.to(device())
    assert torch.equal(ozk.ozk_layernorm(xd, out=xd)[4:], y[4:])
    assert ozk.ozk_layernorm(torch.empty((0, 8), device=device())).shape == (0, 8)


def check_codes(q, scale, y):
    """Codes equal the 64-bit ones except within 1e-9 of a border, where fp64 statistics
    (off by at most (depth + 8) 2^-53 relative, 2e-14 of 127) may fall on the other side."""
    quot, ws = layers.int8_codes(y)
    gs = scale.cpu().numpy()
    assert np.array_equal(np.isnan(gs), np.isnan(ws))
    ok = ~np.isnan(ws)
    np.testing.assert_allclose(gs[ok], ws[ok], rtol=2.0 ** -23, atol=2.0 ** -149)
    diff = q.cpu().numpy().astype(np.int64) - np.rint(quot).astype(np.int64)
    border = np.abs(np.abs(quot - np.floor(quot)) - 0.5) < 1e-9
    # a scale one step of fp32 off moves a quotient by at most 127 * 2^-23
    border |= (gs != ws)[:, None] & (np.abs(np.abs(quot - np.floor(quot)) - 0.5) < 2e-5)
    assert not diff[~border].any(), np.argwhere((diff != 0) & ~border)[:5]
    assert np.abs(diff).max(initial=0) <= 1


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("cols", COLS)
def test_int8quant_rows(kind, cols):
    announce(f"int8quant rows {kind} cols={cols}")
    dtype, rows = TYPES[kind], rows_of(cols)
    x, gamma, beta, _ = row_input(rows, cols, dtype, cols + 2)
    x[1] = 0
    for pad, offset in ((0, 0), (3, 1)):
        xd = padded(x, pad, offset)
        out = padded(torch.full((rows, cols), 99, dtype=torch.int8), pad + 1, offset)
        q, scale = ozk.ozk_int8quant_rows(xd, out=out)
        check_codes(q, scale, host(x))
        assert float(scale[1]) == 0 and not q[1].any()
        q, scale = ozk.ozk_int8quant_rows(xd, norm=True, gamma=gamma.to(device()),
                                          beta=beta.to(device()))
        check_codes(q, scale, layers.layernorm(host(x), host(gamma), host(beta))[0])
        q, scale = ozk.ozk_int8quant_rows(xd, norm=True, eps=0.5)
        check_codes(q, scale, layers.layernorm(host(x), eps=0.5)[0])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("cols", [65, 520, 1030, 2047, 4096, 5000, 8200, 16390])
def test_int8quant_many_rows(kind, cols):
    """The shapes that many rows take; among them rows far from their first value's scale
    (the sums are taken again about the mean), of magnitudes beyond fp32 arithmetic's reach,
    and with quotients on and beside the borders."""
    announce(f"int8quant many rows {kind} cols={cols}")
    dtype, rows = TYPES[kind], 260
    x, gamma, beta, _ = row_input(rows, cols, dtype, cols + 3)
    big = 1e30 if kind in ("float64", "float32", "bfloat16") else 6e4
    x[3, 0] = big                      # the first value alone
    x[4, :] = 1000.0 + x[4] % 1        # far from zero
    x[5] *= 2.0 ** -20
    if kind != "float16":
        x[6] *= 1e36
        x[7] *= 1e-36
    half = torch.arange(cols, dtype=torch.float64) % 255 - 127
    x[8] = (half / 2 + 0.25).to(dtype)
    x[9] = half.to(dtype)
    x[9, 0], x[9, 1:7] = 127, torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, 126.5]).to(dtype)
    x[10] = 0
    x[11, 1] = float("nan")
    xd = padded(x, 1, 3)
    q, scale = ozk.ozk_int8quant_rows(xd)
    check_codes(q, scale, host(x))
    assert q[9, 1:7].tolist() == [0, 2, 2, 0, -2, 126]
    with np.errstate(over="ignore", invalid="ignore"):
        y = layers.layernorm(host(x), host(gamma), host(beta))[0]
        plain = layers.layernorm(host(x))[0]
    # row 3's statistics hang on one value: its others differ from the mean by less than fp64
    # keeps of it, in the reference as well
    keep = [i for i in range(rows) if i != 3]
    q, scale = ozk.ozk_int8quant_rows(xd, norm=True, gamma=gamma.to(device()),
                                      beta=beta.to(device()))
    check_codes(q[keep], scale[keep], y[keep])
    q, scale = ozk.ozk_int8quant_rows(xd, norm=True)
    check_codes(q[keep], scale[keep], plain[keep])


@pytest.mark.parametrize("kind", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("cols", [500, 2000, 16384, 20000])
def test_int8quant_padded_rows(kind, cols):
    """Rows of zeros and, under the norm, of one value (with beta, without, with a beta of zeros),
    beside others: scale and codes as the definition has them."""
    announce(f"int8quant padded rows {kind} cols={cols}")
    dtype, rows = TYPES[kind], 300
    x, gamma, beta, _ = row_input(rows, cols, dtype, cols)
    x[::3] = 0
    x[1::3] = 3.3
    xd, gd, bd = x.to(device()), gamma.to(device()), beta.to(device())
    q, scale = ozk.ozk_int8quant_rows(xd)
    check_codes(q, scale, host(x))
    assert not q[::3].any() and not scale[::3].any()
    zeros = torch.zeros_like(bd)
    for g, b in ((None, None), (gd, None), (gd, zeros), (gd, bd)):
        q, scale = ozk.ozk_int8quant_rows(xd, norm=True, gamma=g, beta=b)
        # (x - mean of one value is 0 exactly; a 64-bit mean may be a rounding off)
        y = layers.layernorm(host(x), None if g is None else host(g),
                             None if b is None else host(b))[0]
        y[::3] = y[1::3] = 0 if b is None else host(b)
        check_codes(q, scale, y)
    # without statistics that are finite, or with a weight that is not, no row is plain
    q, scale = ozk.ozk_int8quant_rows(xd, norm=True, eps=0.0)
    assert torch.isnan(scale[::3]).all() and torch.isnan(scale[1::3]).all() and not q[::3].any()
    gd[cols - 1] = float("inf")
    assert torch.isnan(ozk.ozk_int8quant_rows(xd, norm=True, gamma=gd)[1]).all()


def test_int8quant_zero_rows_take_no_longer():
    """A batch that is half padding costs no more than one without: the least of five times of ten
    calls each, with half as much again for the clock (twice as much was the fault)."""
    announce("int8quant zero rows' time")
    x = torch.randn(4096, 16384, device=device()).bfloat16()
    half = x.clone()
    half[::2] = 0
    q = torch.empty(x.shape, dtype=torch.int8, device=device())
    s = torch.empty(4096, device=device())

    def least(x):
        times = []
        for _ in range(5):
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record()
            for _ in range(10):
                ozk.ozk_int8quant_rows(x, out=q, scale=s)
            e1.record()
            e1.synchronize()
            times.append(e0.elapsed_time(e1))
        return min(times)

    least(x)
    assert least(half) < 1.5 * least(x)


def test_int8quant_rows_edges():
    """NaN, Inf, fp64 values past fp32's range, values below every fp32 scale, subnormal
    scales, ties to even; what stands behind a row's end stays."""
    announce("int8quant edges")
    x = torch.zeros(8, 100, dtype=torch.float64)
    x[0, 3], x[1, 99] = float("nan"), -float("inf")
    x[2, :] = 1e60
    x[3, 0] = 1e-60
    x[4, 0], x[4, 1] = 127 * 1.4 * 2.0 ** -149, 2.0 ** -149
    x[5, 0], x[5, 1], x[5, 2], x[5, 3] = 127.0, 0.5, 1.5, -2.5
    x[6] = torch.linspace(-3, 3, 100, dtype=torch.float64)
    buf = torch.full((8, 104), 55, dtype=torch.int8, device=device())
    q, scale = ozk.ozk_int8quant_rows(x.to(device()), out=buf[:, :100])
    check_codes(q, scale, x.numpy())
    s = scale.cpu()
    assert torch.isnan(s[:3]).all() and not q[:3].any()
    assert s[3] == 0 and not q[3].any()
    assert s[4] > 0 and q[4, 0] == 127
    assert q[5, :4].tolist() == [127, 0, 2, -2]
    assert (buf[:, 100:] == 55).all()
    # a row whose statistics or weights are not finite
    w = torch.ones(100, dtype=torch.float64)
    w[7] = float("inf")
    q, scale = ozk.ozk_int8quant_rows(x[5:7].to(device()), norm=True, gamma=w.to(device()))
    assert torch.isnan(scale).all() and not q.any()
    q, scale = ozk.ozk_int8quant_rows(x[:2].to(device()), norm=True)
    assert torch.isnan(scale).all() and not q.any()


# ------------------------------------------------------------------ int8 linear layer
def int8_case(m, n, k, kind, seed, extreme=False):
    rng = np.random.default_rng(seed)
    x, w = ozk_inputs.int8_matrix(rng, (m, k)), ozk_inputs.int8_matrix(rng, (n, k))
    if extreme:
        x[:], w[:] = -128, -128
    dtype = TYPES[kind]
    sx = torch.from_numpy(np.exp(rng.standard_normal(m)) / 127).float()
    sw = torch.from_numpy(np.exp(0.3 * rng.standard_normal(n)) / 127 / np.sqrt(k)).float()
    bias = torch.from_numpy(rng.standard_normal(n)).to(dtype)
    res = torch.from_numpy(rng.standard_normal((m, n))).to(dtype)
    return torch.from_numpy(x), sx, torch.from_numpy(w), sw, bias, res


def check_linear(got, x, sx, w, sw, bias, name, res):
    """z: one rounding of the sum, one for each scale and the bias.  An activation stretches an
    error by at most 1.13 and adds 16 roundings of its own (exp and erfc are within a few, the
    argument of either is rounded twice, |z| d/dz of both factors is below 2)."""
    z = layers.int8_sums(x.numpy(), w.numpy()) * host(sx)[:, None] * host(sw)
    ez = 3 * U32 * np.abs(z)
    if bias is not None:
        z = z + host(bias)
        ez = ez + U32 * np.abs(z)
    want = layers.act(z, name)
    err = 1.13 * ez * 1.01 + (16 * U32 * np.abs(z) if name not in ("none", "relu") else 0)
    if res is not None:
        want = want + host(res)
        err = err + U32 * np.abs(want)
    assert_near(host(got), want, err + half_step(got.dtype) * (np.abs(want) + err)
                + tiny(got.dtype), f"int8linear {name}")


# one row to several tiles of rows; columns and K around the tiles, odd and ragged; K of one
# value, below a step, and long
LINEAR = [(1, 1, 1), (1, 16, 64), (1, 700, 1000), (2, 33, 129), (7, 4100, 257), (16, 256, 4096),
          (17, 130, 1001), (31, 65, 128), (33, 1000, 300), (48, 272, 2048), (64, 128, 128),
          (65, 129, 256), (100, 515, 383), (128, 256, 512), (130, 300, 1024), (200, 96, 5000),
          (256, 256, 256), (300, 520, 384), (513, 257, 640), (1000, 1030, 130), (3, 48, 30000),
          (128, 128, 16384), (700, 2050, 1024),
          # enough tiles of 256 x 256 for every compute unit: K whole, ending in a step, odd
          (3000, 4500, 272), (2900, 4600, 384), (3000, 4500, 131)]


@pytest.mark.parametrize("m,n,k", LINEAR)
@pytest.mark.parametrize("kind", ["float32", "float16", "bfloat16"])
def test_int8linear(m, n, k, kind):
    announce(f"int8linear m={m} n={n} k={k} {kind}")
    x, sx, w, sw, bias, res = int8_case(m, n, k, kind, m * 7 + n * 3 + k)
    d = device()
    for name, b, r, pad in (("none", None, None, 0), ("gelu", bias, res, 0),
                            ("silu", bias, None, 3), ("gelu_tanh", None, res, 5),
                            ("relu", bias, res, 16)):
        buf = torch.full((m, n + 2 * pad), 3.0, dtype=TYPES[kind], device=d)
        got = ozk.ozk_int8linear(
            padded(x, pad, pad % 16), sx.to(d), padded(w, pad, 2 * pad % 16), sw.to(d),
            bias=None if b is None else b.to(d), act=name,
            residual=None if r is None else padded(r, pad), out=buf[:, :n])
        check_linear(got, x, sx, w, sw, b, name, r)
        assert (buf[:, n:] == 3.0).all()


@pytest.mark.parametrize("name", layers.ACTS[1:])
@pytest.mark.parametrize("kind", ["float32", "float16", "bfloat16"])
def test_int8linear_activation_digits(kind, name):
    """The activations of z = bias (zero codes), relative to the result however small it is.  In
    units of 2^-24, for fp32: gelu and silu 12 (exp2 within two, its argument's remainder, the
    reciprocal, the polynomial two or three, three or four products and the fit's quarter);
    gelu_tanh's exponent v is rounded six times before, 6 |v| more.  16-bit types: 2^-16 from the
    shorter fit and exp2's argument (gelu), 8 |v| and 12 from v and exp2's argument (the others).
    Results below 2^-119 may come as zero."""
    announce(f"int8linear activation digits {kind} {name}")
    dtype = TYPES[kind]
    z = np.concatenate([np.linspace(-13.5, 13.5, 5001), -np.exp(np.linspace(-30, 4.4, 900)),
                        np.exp(np.linspace(-30, 4.4, 900)), [0.0, 1.0, -1.0, 1e4, -1e4, 6e4]])
    z = torch.from_numpy(z).to(dtype)
    hz = host(z)
    n = hz.size
    for m in (1, 20, 130):   # rows of two kernels for few rows, one of tiles
        x = torch.zeros((m, 32), dtype=torch.int8, device=device())
        w = torch.ones((n, 32), dtype=torch.int8, device=device())
        got = host(ozk.ozk_int8linear(x, torch.ones(m, device=device()), w,
                                      torch.ones(n, device=device()), bias=z.to(device()),
                                      act=name, dtype=dtype))
        assert (got == got[0]).all()
        want = layers.act(hz, name)
        v = np.minimum(2 * np.sqrt(2 / np.pi) * np.abs(hz + 0.044715 * hz ** 3), 100)
        v = v if name == "gelu_tanh" else np.minimum(np.abs(hz), 100)
        if name == "relu":
            rel = 0
        elif kind == "float32":
            rel = (12 + (6 * v if name == "gelu_tanh" else 0)) * U32
        else:
            rel = 2.0 ** -16 if name == "gelu" else (12 + 8 * v) * U32
        err = rel * np.abs(want) + 2.0 ** -119
        assert_near(got[0], want, err + half_step(dtype) * (np.abs(want) + err) + tiny(dtype),
                    f"{name} m={m}")
    far = torch.tensor([float("inf"), float("nan"), 3e38, -3e38], dtype=torch.float32).to(dtype)
    got = ozk.ozk_int8linear(x, torch.ones(m, device=device()), w[:4],
                             torch.ones(4, device=device()), bias=far.to(device()), act=name,
                             dtype=dtype)[0].double().cpu()
    assert got[0] == np.inf and torch.isnan(got[1]) and got[2] == far[2].double()
    assert got[3] == 0 or kind == "float16"   # (there -3e38 is -Inf: the formula's Inf times 0)


@pytest.mark.parametrize("m", [1, 20, 130])
def test_int8linear_longest_k(m):
    """K = 131071 of (-128)(-128): every sum is 2147467264, the largest that int32 must hold."""
    announce(f"int8linear longest k m={m}")
    x, sx, w, sw, bias, res = int8_case(m, 48, 131071, "float32", 9, extreme=True)
    d = device()
    got = ozk.ozk_int8linear(x.to(d), sx.to(d), w.to(d), sw.to(d), dtype=torch.float32)
    check_linear(got, x, sx, w, sw, None, "none", None)


def test_int8linear_edges():
    """Nothing to do; the residual in place; NaN scales touch their row or column only; codes
    of -128; the outputs of a batch's rows do not depend on the rows beside them."""
    announce("int8linear edges")
    d = device()
    x, sx, w, sw, bias, res = [t.to(d) for t in int8_case(70, 90, 300, "bfloat16", 4)]
    want = ozk.ozk_int8linear(x, sx, w, sw, bias=bias, act="gelu", residual=res)
    c = res.clone()
    assert ozk.ozk_int8linear(x, sx, w, sw, bias=bias, act="gelu", residual=c, out=c) is c
    assert torch.equal(c, want)
    for i in (0, 33, 69):
        one = ozk.ozk_int8linear(x[i:i + 1], sx[i:i + 1], w, sw, bias=bias, act="gelu",
                                 residual=res[i:i + 1])
        assert torch.equal(one, want[i:i + 1])
    s2 = sx.clone()
    s2[3] = float("nan")
    t2 = sw.clone()
    t2[5] = float("nan")
    got = ozk.ozk_int8linear(x, s2, w, t2, bias=bias, act="gelu", residual=res)
    nan = torch.isnan(got)
    assert nan[3].all() and nan[:, 5].all() and int(nan.sum()) == 90 + 70 - 1
    assert torch.equal(got[~nan], want[~nan])
    assert ozk.ozk_int8linear(x[:0], sx[:0], w, sw).shape == (0, 90)
    assert ozk.ozk_int8linear(x, sx, w[:0], sw[:0]).shape == (70, 0)


# ------------------------------------------------------------------ fp64 product, epilogue
def act_error(z, y):
    """16 roundings of the function's value, and of |z| where its argument is rounded."""
    return 16 * U64 * (np.abs(y) + np.abs(z)) + 2.0 ** -1074


@pytest.mark.parametrize("m,n,k,r,scaling", [(1, 1, 1, 14, "max"), (3, 65, 40, 14, "norm"),
                                             (64, 64, 64, 14, "max"), (70, 130, 129, 16, "norm"),
                                             (257, 66, 300, 18, "max"), (33, 300, 1000, 20, "max")])
def test_dgemm_epilogue(m, n, k, r, scaling):
    announce(f"dgemm epilogue m={m} n={n} k={k} r={r} {scaling}")
    a, b = ozk_inputs.gemm_operands(m, n, k, seed=m + n + k, dist="phi", phi=0.5)
    rng = np.random.default_rng(m)
    bias, res = rng.standard_normal(n), rng.standard_normal((m, n))
    prod = ozaki2.dgemm(a, b, r, scaling=scaling)
    for name, bi, re, pad in (("none", None, None, 0), ("none", bias, res, 1),
                              ("relu", bias, None, 0), ("gelu", bias, res, 3),
                              ("gelu_tanh", None, res, 0), ("silu", bias, res, 2)):
        z = torch.full((m, n + pad), 5.0, dtype=torch.float64, device=device())
        c = torch.full((m, n + 2 * pad), 5.0, dtype=torch.float64, device=device())
        ozk.ozk_dgemm_epilogue(
            padded(torch.from_numpy(a), pad), padded(torch.from_numpy(b), pad), r,
            bias=None if bi is None else to_dev(bi), act=name,
            residual=None if re is None else padded(torch.from_numpy(re), pad),
            scaling=scaling, preact=z[:, :n], out=c[:, :n])
        wz = prod if bi is None else prod + bi
        np.testing.assert_array_equal(host(z[:, :n]), wz)     # the same roundings: bit for bit
        wy = layers.act(wz, name)
        want = wy if re is None else wy + re
        tol = act_error(wz, wy) if name not in ("none", "relu") else np.zeros_like(wz)
        # act(z) + residual is rounded once here and once in the reference, which is fp64 too:
        # two roundings of the sum lie between them where act(z) differs at all
        if tol.any():
            tol = tol + 2 * U64 * np.abs(want)
        assert_near(host(c[:, :n]), want, tol, name)
        assert (z[:, n:] == 5.0).all() and (c[:, n:] == 5.0).all()


def test_dgemm_epilogue_equals_dgemm():
    """Without an epilogue the bits of ozk_dgemm_ex; the residual in place; NaN and Inf."""
    announce("dgemm epilogue = dgemm")
    a, b = ozk_inputs.gemm_operands(130, 200, 513, seed=2, dist="phi", phi=4.0)
    a[7, 3] = np.nan
    da, db = to_dev(a), to_dev(b)
    want = ozk.ozk_dgemm_ex(da, db, 16, "norm")
    got = ozk.ozk_dgemm_epilogue(da, db, 16, scaling="norm")
    assert torch.equal(got.view(torch.int64), want.view(torch.int64))
    assert torch.isnan(got[7]).all() and not torch.isnan(got[8]).any()
    res = to_dev(np.random.default_rng(0).standard_normal((130, 200)))
    apart = ozk.ozk_dgemm_epilogue(da, db, 16, act="silu", residual=res)
    inplace = ozk.ozk_dgemm_epilogue(da, db, 16, act="silu", residual=res, out=res)
    assert inplace is res
    assert torch.equal(apart.view(torch.int64), res.view(torch.int64))
    assert ozk.ozk_dgemm_epilogue(da[:0], db, 14).shape == (0, 200)


# inner and outer sizes on both sides of what the kernels for small products take, one and
# several tiles of each shape, padded and whole rows of residues
@pytest.mark.parametrize("m,n,k,r", [(130, 65, 2047, 16), (65, 130, 2049, 16), (40, 70, 5000, 14),
                                     (1500, 2050, 1001, 16), (700, 640, 2500, 15),
                                     (2048, 1537, 256, 14), (300, 5000, 130, 20), (1, 300, 700, 14),
                                     (64, 100, 8192, 16)])
@pytest.mark.parametrize("scaling", ["max", "norm"])
def test_dgemm_epilogue_bits_of_dgemm(m, n, k, r, scaling):
    """The product inside the epilogue and both products of its gradient have the bits of
    ozk_dgemm_ex on the same operands."""
    announce(f"dgemm epilogue bits m={m} n={n} k={k} r={r} {scaling}")
    a, b = [to_dev(v) for v in ozk_inputs.gemm_operands(m, n, k, seed=m + n + k, dist="phi",
                                                        phi=0.5)]
    rng = np.random.default_rng(n)
    dc, res = to_dev(rng.standard_normal((m, n))), to_dev(rng.standard_normal((m, n)))
    got = ozk.ozk_dgemm_epilogue(a, b, r, residual=res, scaling=scaling)
    assert torch.equal(got, ozk.ozk_dgemm_ex(a, b, r, scaling) + res)
    da, db, dbias = ozk.ozk_dgemm_epilogue_grad(dc, a, b, r, scaling=scaling)
    assert torch.equal(da, ozk.ozk_dgemm_ex(dc, to_dev(host(b).T.copy()), r, scaling))
    assert torch.equal(db, ozk.ozk_dgemm_ex(to_dev(host(a).T.copy()), dc, r, scaling))
    assert_near(host(dbias), host(dc).sum(0),
                (m // 16 + 80) * U64 * np.abs(host(dc)).sum(0) + 1e-300, "dbias")


@pytest.mark.parametrize("m,n,k", [(2090, 70, 1000), (2100, 70, 1000), (70, 2090, 1000),
                                   (70, 2100, 1000), (130000, 40, 256), (132000, 40, 256),
                                   (40, 130000, 256), (40, 132000, 256)])
def test_dgemm_epilogue_where_operands_stop_being_small(m, n, k):
    """2^21 values, or 2^25 in lines of 256: the bits of ozk_dgemm_ex on either side."""
    announce(f"dgemm epilogue small or not m={m} n={n} k={k}")
    g = torch.Generator(device=device()).manual_seed(m + n)
    a = torch.randn(m, k, generator=g, device=device(), dtype=torch.float64)
    b = torch.randn(k, n, generator=g, device=device(), dtype=torch.float64)
    for scaling in ("max", "norm"):
        assert torch.equal(ozk.ozk_dgemm_epilogue(a, b, 14, scaling=scaling),
                           ozk.ozk_dgemm_ex(a, b, 14, scaling))


@pytest.mark.parametrize("n", [4100, 4200])
def test_dgemm_epilogue_grad_where_columns_stop_being_small(n):
    """2^23 values in columns of 2040, and G's rows past any small line: both products' bits."""
    m, k = 2040, 70
    announce(f"dgemm epilogue grad small or not n={n}")
    g = torch.Generator(device=device()).manual_seed(n)
    new = lambda *s: torch.randn(*s, generator=g, device=device(), dtype=torch.float64)
    dc, a, b = new(m, n), new(m, k), new(k, n)
    da, db, _ = ozk.ozk_dgemm_epilogue_grad(dc, a, b, 14)
    assert torch.equal(da, ozk.ozk_dgemm_ex(dc, b.t().contiguous(), 14))
    assert torch.equal(db, ozk.ozk_dgemm_ex(a.t().contiguous(), dc, 14))


def test_dgemm_epilogue_columns_past_a_launch():
    """One row against 2^26 columns, 16 moduli: as many of the smaller tiles as a launch of 512
    threads a tile cannot take.  Small integers, so every product is exact."""
    m, n, k, r = 1, 1 << 26, 1, 16
    announce(f"dgemm epilogue m={m} n={n} k={k} r={r}")
    need = ozk.ozk_dgemm_epilogue_workspace_size(m, n, k, r) + 32 * n
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of device memory")
    b = (torch.arange(n, device=device()) % 1021 - 510).double()[None]
    a = torch.full((1, 1), 3.0, dtype=torch.float64, device=device())
    c = ozk.ozk_dgemm_epilogue(a, b, r, act="relu")
    assert torch.equal(c, (3 * b).clamp(min=0))
    del c
    torch.cuda.empty_cache()   # the workspace's 137 GB


def test_dgemm_epilogue_rows_past_a_launch():
    """2^24 rows and some, a workgroup a row: deconstructed by more than one launch."""
    m, n, k, r = (1 << 24) + 5, 2, 3, 14
    announce(f"dgemm epilogue m={m} n={n} k={k} r={r}")
    need = ozk.ozk_dgemm_epilogue_workspace_size(m, n, k, r) + 64 * m
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of device memory")
    i = torch.arange(m, device=device())
    a = torch.stack([i % 1021 - 510, i % 7, -(i % 64)], 1).double()   # exact products and sums
    b = torch.tensor([[3.0, -1.0], [100.0, 7.0], [5.0, 0.5]], device=device(), dtype=torch.float64)
    want = (a[:, :, None] * b[None]).sum(1)
    assert torch.equal(ozk.ozk_dgemm_epilogue(a, b, r), want)
    assert torch.equal(ozk.ozk_dgemm_ex(a, b, r), want)
    del a, want, i
    torch.cuda.empty_cache()


@pytest.mark.parametrize("scaling", ["max", "norm"])
def test_dgemm_epilogue_grad_many_long_rows(scaling):
    """More than 65535 rows of dC, each past the 32768 values that a workgroup holds: the rows of
    dA are those of a few rows alone, bit for bit."""
    m, n, k, r = 65600, 32800, 2, 8
    announce(f"dgemm epilogue grad m={m} n={n} k={k} r={r} {scaling}")
    need = ozk.ozk_dgemm_epilogue_grad_workspace_size(m, n, k, r) + 10 * m * n
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of device memory")
    g = torch.Generator(device=device()).manual_seed(3)
    dc = torch.randn(m, n, generator=g, device=device(), dtype=torch.float64)
    b = torch.randn(k, n, generator=g, device=device(), dtype=torch.float64)
    a = torch.zeros(m, k, device=device(), dtype=torch.float64)
    grad = lambda lo, hi: ozk.ozk_dgemm_epilogue_grad(
        dc[lo:hi], a[lo:hi], b, r, scaling=scaling, need_db=False, need_dbias=False)[0]
    da = grad(0, m)
    for lo, hi in ((0, 70), (65500, 65600)):
        assert torch.equal(da[lo:hi], grad(lo, hi))
    del dc, da
    torch.cuda.empty_cache()


def test_dgemm_epilogue_grad_nonfinite():
    """A line with Inf or NaN spoils the outputs it touches, in the small kernels too."""
    announce("dgemm epilogue grad nonfinite")
    rng = np.random.default_rng(5)
    a, b = rng.standard_normal((70, 40)), rng.standard_normal((40, 90))
    dc = rng.standard_normal((70, 90))
    dc[3, 5] = np.inf
    a[9, 2] = np.nan
    da, db, dbias = ozk.ozk_dgemm_epilogue_grad(to_dev(dc), to_dev(a), to_dev(b), 16)
    na, nb = torch.isnan(da), torch.isnan(db)
    assert na[3].all() and int(na.sum()) == 40
    assert nb[:, 5].all() and nb[2].all() and int(nb.sum()) == 40 + 90 - 1
    assert torch.isinf(dbias[5]) and int(torch.isinf(dbias).sum()) == 1


@pytest.mark.parametrize("k", [1, 127, 128, 129, 255, 256, 257, 511, 512, 513])
@pytest.mark.parametrize("scaling", ["max", "norm"])
def test_dgemm_epilogue_line_lengths(k, scaling):
    """Both sides of the steps that a thread holds of a line; lines of zeros, with an Inf, a NaN,
    and far magnitudes.  The gradient's products run over n = k and m = k."""
    announce(f"dgemm epilogue line lengths k={k} {scaling}")
    rng = np.random.default_rng(k)
    a, b = rng.standard_normal((37, k)), rng.standard_normal((k, 50))
    a[3] = 0.0
    b[:, 5] = 0.0
    a[7] *= 1e250
    b[:, 9] *= 1e-250
    a[11, k - 1], b[k // 2, 13] = np.inf, np.nan
    same = lambda x, y: np.testing.assert_array_equal(host(x), host(y))
    ad, bd = padded(torch.from_numpy(a), 1, 1), padded(torch.from_numpy(b), 3)
    same(ozk.ozk_dgemm_epilogue(ad, bd, 16, scaling=scaling),
         ozk.ozk_dgemm_ex(ad, bd, 16, scaling=scaling))
    # dA: dC (37 x k) times rows of B (50 x k); dB: columns of A (k x 37) against dC (k x 50)
    da, _, _ = ozk.ozk_dgemm_epilogue_grad(ad, to_dev(rng.standard_normal((37, 50))),
                                           to_dev(b.T), 16, scaling=scaling)
    same(da, ozk.ozk_dgemm_ex(ad, bd, 16, scaling=scaling))
    _, db, _ = ozk.ozk_dgemm_epilogue_grad(bd, to_dev(a.T), to_dev(rng.standard_normal((37, 50))),
                                           16, scaling=scaling)
    same(db, ozk.ozk_dgemm_ex(ad, bd, 16, scaling=scaling))


@pytest.mark.parametrize("m", [1, 15, 64, 65, 1024, 1025, 2500])
def test_dgemm_epilogue_grad_bias(m):
    """The bias's gradient alone, and G where all columns are short: m / 16 + 48 roundings of the
    sum beside 64 of G."""
    announce(f"dgemm epilogue grad bias m={m}")
    rng = np.random.default_rng(m)
    for n, act in ((1, "silu"), (17, "gelu"), (300, "none")):
        dc, z = rng.standard_normal((m, n)), 2 * rng.standard_normal((m, n))
        a, b = to_dev(rng.standard_normal((m, 5))), to_dev(rng.standard_normal((5, n)))
        _, _, dbias = ozk.ozk_dgemm_epilogue_grad(
            padded(torch.from_numpy(dc), 2), a, b, 14, act=act, need_da=False, need_db=False,
            preact=padded(torch.from_numpy(z), 1) if act != "none" else None)
        g = dc * layers.slope(z, act)
        tol = (64 * U64 * np.abs(dc) * (1 + z * z)).sum(0)
        assert_near(host(dbias), g.sum(0), tol + (m // 16 + 48) * U64 * np.abs(g).sum(0), "dbias")
        again = ozk.ozk_dgemm_epilogue_grad(to_dev(dc), a, b, 14, act=act, preact=to_dev(z))
        assert torch.equal(again[2], dbias)


def test_dgemm_epilogue_large_arguments():
    """Pre-activations far out: the activations and slopes settle without NaN."""
    announce("dgemm epilogue large arguments")
    z = np.array([[-1e300, -1e3, -40.0, -8.0, -1e-300, 0.0, 1e-300, 8.0, 40.0, 1e3, 1e300]])
    one = np.ones((1, 1))
    for name in layers.ACTS[1:]:
        c = host(ozk.ozk_dgemm_epilogue(to_dev(one), to_dev(z), 20, act=name))
        with np.errstate(over="ignore", invalid="ignore"):
            want = np.where(z > 1e2, z, np.where(z < -1e2, 0.0, layers.act(z, name)))
        assert_near(c, want, act_error(np.where(np.abs(z) > 1e2, 0, z), want), name)
        g = host(ozk.ozk_dgemm_epilogue_grad(to_dev(np.ones_like(z)), to_dev(one), to_dev(z), 14,
                                             preact=to_dev(z), act=name, need_da=False,
                                             need_db=False)[2])[None]
        with np.errstate(over="ignore", invalid="ignore"):
            ws = np.where(z > 1e2, 1.0, np.where(z < -1e2, 0.0, layers.slope(z, name)))
        assert_near(g, ws, 64 * U64 * np.maximum(1, np.where(np.abs(z) > 1e2, 0, z) ** 2), name)


@pytest.mark.parametrize("m,n,k,r,scaling", [(1, 1, 1, 14, "max"), (64, 64, 64, 14, "norm"),
                                             (70, 130, 129, 16, "norm"), (257, 66, 300, 15, "max"),
                                             (300, 1000, 33, 20, "max")])
def test_dgemm_epilogue_grad_products(m, n, k, r, scaling):
    """Without an activation G is dC: both products bit for bit the oracle's, whose left and
    right operands have the widths of A and B; dbias within (m / 16 + 32) roundings."""
    announce(f"dgemm epilogue grad m={m} n={n} k={k} r={r} {scaling}")
    a, b = ozk_inputs.gemm_operands(m, n, k, seed=m + n, dist="phi", phi=0.5)
    dc = np.random.default_rng(k).standard_normal((m, n))
    for pad in (0, 3):
        da, db, dbias = ozk.ozk_dgemm_epilogue_grad(
            padded(torch.from_numpy(dc), pad), padded(torch.from_numpy(a), pad),
            padded(torch.from_numpy(b), pad), r, scaling=scaling)
        np.testing.assert_array_equal(host(da), ozaki2.dgemm(dc, np.ascontiguousarray(b.T), r,
                                                             scaling=scaling))
        np.testing.assert_array_equal(host(db), ozaki2.dgemm(np.ascontiguousarray(a.T), dc, r,
                                                             scaling=scaling))
        assert_near(host(dbias), dc.sum(0), (m // 16 + 48) * U64 * np.abs(dc).sum(0) + 1e-300,
                    "dbias")


@pytest.mark.parametrize("name", layers.ACTS)
@pytest.mark.parametrize("m,n,k", [(50, 70, 90), (300, 129, 64)])
def test_dgemm_epilogue_grad_activations(m, n, k, name):
    """Against the formula in 64 bits.  G is off by 64 roundings (the slope's factors); a
    product's inner sums by that, by their own rounding in the reference, and by the scaled
    integers: half a unit of 2^-P of the line's maximum per term, P >= 44 for r = 16."""
    announce(f"dgemm epilogue grad {name} m={m} n={n} k={k}")
    rng = np.random.default_rng(m + n)
    a, b = rng.standard_normal((m, k)), rng.standard_normal((k, n))
    dc, z = rng.standard_normal((m, n)), 2 * rng.standard_normal((m, n))
    da, db, dbias = ozk.ozk_dgemm_epilogue_grad(to_dev(dc), to_dev(a), to_dev(b), 16,
                                                preact=to_dev(z), act=name)
    g = dc * layers.slope(z, name)
    eg = 64 * U64 * np.abs(dc) * (1 + z * z)

    def tol(left, right, eleft, eright):
        inner = left.shape[1]
        scaled = inner * 2.0 ** -44 * np.abs(left).max(1)[:, None] * np.abs(right).max(0)
        return (eleft @ np.abs(right) + np.abs(left) @ eright
                + 2 * inner * U64 * (np.abs(left) @ np.abs(right)) + scaled)

    assert_near(host(da), g @ b.T, tol(g, b.T, eg, np.zeros_like(b.T)), "dA")
    assert_near(host(db), a.T @ g, tol(a.T, g, np.zeros_like(a.T), eg), "dB")
    assert_near(host(dbias), g.sum(0), eg.sum(0) + 400 * U64 * np.abs(g).sum(0), "dbias")


@pytest.mark.parametrize("name", layers.ACTS)
@pytest.mark.parametrize("m,n,k", [(1025, 130, 20), (1500, 300, 33), (4200, 70, 9)])
def test_dgemm_epilogue_grad_long_activations(m, n, k, name):
    """More rows than the short kernel of G takes: G goes into both products.  Chunks of 16 rows,
    the last of one or of twelve, and of 17; padded dC and Z.  Bounds as above."""
    announce(f"dgemm epilogue grad long {name} m={m} n={n} k={k}")
    rng = np.random.default_rng(m + n)
    a, b = rng.standard_normal((m, k)), rng.standard_normal((k, n))
    dc, z = rng.standard_normal((m, n)), 2 * rng.standard_normal((m, n))
    da, db, dbias = ozk.ozk_dgemm_epilogue_grad(
        padded(torch.from_numpy(dc), 3), to_dev(a), to_dev(b), 16,
        preact=padded(torch.from_numpy(z), 1), act=name)
    g = dc * layers.slope(z, name)
    eg = 64 * U64 * np.abs(dc) * (1 + z * z)

    def tol(left, right, eleft, eright):
        inner = left.shape[1]
        scaled = inner * 2.0 ** -44 * np.abs(left).max(1)[:, None] * np.abs(right).max(0)
        return (eleft @ np.abs(right) + np.abs(left) @ eright
                + 2 * inner * U64 * (np.abs(left) @ np.abs(right)) + scaled)

    assert_near(host(da), g @ b.T, tol(g, b.T, eg, np.zeros_like(b.T)), "dA")
    assert_near(host(db), a.T @ g, tol(a.T, g, np.zeros_like(a.T), eg), "dB")
    assert_near(host(dbias), g.sum(0), eg.sum(0) + (m // 16 + 80) * U64 * np.abs(g).sum(0), "dbias")


def test_dgemm_epilogue_grad_is_the_difference_quotient():
    """The gradient of sum(dC * C) for C = gelu(A B + bias), against central differences of
    the library's own forward: h = 2^-16 leaves h^2 |f'''| / 6 (|f'''| below 400 at these
    sizes: 1.6e-8) and 2^-52 |f| / h (|f| < 1000: 1.5e-8)."""
    announce("dgemm epilogue grad differences")
    rng = np.random.default_rng(6)
    a, b, bias = rng.standard_normal((5, 4)), rng.standard_normal((4, 6)), rng.standard_normal(6)
    dc = rng.standard_normal((5, 6))
    z = torch.empty((5, 6), dtype=torch.float64, device=device())

    def f(a, b, bias):
        return float((dc * host(ozk.ozk_dgemm_epilogue(to_dev(a), to_dev(b), 20, act="gelu",
                                                       bias=to_dev(bias)))).sum())

    ozk.ozk_dgemm_epilogue(to_dev(a), to_dev(b), 20, act="gelu", bias=to_dev(bias), preact=z)
    grads = ozk.ozk_dgemm_epilogue_grad(to_dev(dc), to_dev(a), to_dev(b), 20, preact=z,
                                        act="gelu")
    h = 2.0 ** -16
    for which, (v, g) in enumerate(zip((a, b, bias), grads)):
        for at in ((0,), (3,)) if v.ndim == 1 else ((0, 0), (3, 2)):
            e = np.zeros_like(v)
            e[at] = h
            up = [x + e if i == which else x for i, x in enumerate((a, b, bias))]
            dn = [x - e if i == which else x for i, x in enumerate((a, b, bias))]
            assert abs((f(*up) - f(*dn)) / (2 * h) - host(g)[at]) < 1e-7


def test_dgemm_epilogue_grad_parts():
    announce("dgemm epilogue grad parts")
    rng = np.random.default_rng(8)
    a, b = to_dev(rng.standard_normal((40, 30))), to_dev(rng.standard_normal((30, 50)))
    dc, z = to_dev(rng.standard_normal((40, 50))), to_dev(rng.standard_normal((40, 50)))
    whole = ozk.ozk_dgemm_epilogue_grad(dc, a, b, 14, preact=z, act="silu")
    for i in range(3):
        need = dict(need_da=i == 0, need_db=i == 1, need_dbias=i == 2)
        part = ozk.ozk_dgemm_epilogue_grad(dc, a, b, 14, preact=z, act="silu", **need)
        assert [p is None for p in part] == [j != i for j in range(3)]
        assert torch.equal(part[i], whole[i])
    # sums of no terms
    da, db, dbias = ozk.ozk_dgemm_epilogue_grad(dc[:0], a[:0], b, 14, preact=z[:0], act="silu")
    assert da.shape == (0, 30) and not db.any() and not dbias.any() and db.shape == (30, 50)
    wide = torch.full((40, 35), 2.0, dtype=torch.float64, device=device())
    da, db, dbias = ozk.ozk_dgemm_epilogue_grad(dc[:, :0], a, b[:, :0], 14, da=wide[:, :30])
    assert not da.any() and (wide[:, 30:] == 2.0).all() and dbias.shape == (0,)


# ------------------------------------------------------------------ together
def block(x, p, dtype):
    """A pre-norm feed-forward block on int8 codes: x + W2 gelu(W1 norm(x) + b1) + b2."""
    q, s = ozk.ozk_int8quant_rows(x, norm=True, gamma=p["gamma"], beta=p["beta"])
    h = ozk.ozk_int8linear(q, s, p["w1"], p["s1"], bias=p["b1"], act="gelu", dtype=dtype)
    q, s = ozk.ozk_int8quant_rows(h)
    return ozk.ozk_int8linear(q, s, p["w2"], p["s2"], bias=p["b2"], residual=x, dtype=dtype)


def block_weights(width, hidden, dtype, seed):
    rng = np.random.default_rng(seed)
    w = {"gamma": 1 + 0.1 * rng.standard_normal(width), "beta": 0.1 * rng.standard_normal(width),
         "b1": 0.1 * rng.standard_normal(hidden), "b2": 0.1 * rng.standard_normal(width)}
    p = {k: torch.from_numpy(v).to(dtype).to(device()) for k, v in w.items()}
    for name, shape in (("1", (hidden, width)), ("2", (width, hidden))):
        q, s = ozk.ozk_int8quant_rows(to_dev(rng.standard_normal(shape) / np.sqrt(shape[1])))
        p["w" + name], p["s" + name] = q, s
    return p


@pytest.mark.parametrize("tokens", [1, 9, 200])
def test_block_on_codes(tokens):
    """The block step by step: each step's output against the plain form of that step on the
    step's own inputs, so that a code's rounding does not enter twice."""
    announce(f"int8 block tokens={tokens}")
    dtype = torch.bfloat16
    p = block_weights(264, 1040, dtype, 1)
    x = torch.from_numpy(np.random.default_rng(2).standard_normal((tokens, 264))).to(dtype)
    xd = x.to(device())
    q, s = ozk.ozk_int8quant_rows(xd, norm=True, gamma=p["gamma"], beta=p["beta"])
    check_codes(q, s, layers.layernorm(host(x), host(p["gamma"]), host(p["beta"]))[0])
    h = ozk.ozk_int8linear(q, s, p["w1"], p["s1"], bias=p["b1"], act="gelu")
    check_linear(h, q.cpu(), s, p["w1"].cpu(), p["s1"], p["b1"], "gelu", None)
    q2, s2 = ozk.ozk_int8quant_rows(h)
    check_codes(q2, s2, host(h))
    y = block(xd, p, dtype)
    check_linear(y, q2.cpu(), s2, p["w2"].cpu(), p["s2"], p["b2"], "none", xd)


def test_block_captured_and_on_streams():
    """The serving block captured into a graph and replayed with new tokens between eager
    calls, and eager on two streams at once, gives the eager bits every time."""
    announce("int8 block captured")
    dtype = torch.bfloat16
    p = block_weights(512, 1536, dtype, 3)
    rng = np.random.default_rng(4)
    batches = [torch.from_numpy(rng.standard_normal((24, 512))).to(dtype).to(device())
               for _ in range(4)]
    want = [block(x, p, dtype) for x in batches]
    static = batches[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(static, p, dtype)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(static, p, dtype)
    for turn in range(3):
        for x, y in zip(batches, want):
            static.copy_(x)
            graph.replay()
            assert torch.equal(block(x, p, dtype), y)
            torch.cuda.synchronize()
            assert torch.equal(out, y)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            got.append(block(batches[i % 4], p, dtype))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 4])


def train_step(x, dy, gamma, beta, w, b):
    """Layer norm, a gelu layer with the input as its residual, and all gradients, in fp64."""
    y, mean, rstd = ozk.ozk_layernorm(x, gamma, beta, stats=True)
    z = torch.empty_like(dy)
    c = ozk.ozk_dgemm_epilogue(y, w, 16, bias=b, act="gelu", residual=x, preact=z,
                               scaling="norm")
    dyn, dw, db = ozk.ozk_dgemm_epilogue_grad(dy, y, w, 16, preact=z, act="gelu", scaling="norm")
    dx, dgamma, dbeta = ozk.ozk_layernorm_backward(dyn, x, gamma, mean, rstd)
    return c, dx + dy, dgamma, dbeta, dw, db


def test_training_step():
    """Against the same chain in 64 bits: a relative 1e-11 leaves room for the widths of the
    scaled integers (2^-44 of the line's maximum, inner sums of at most 200 terms)."""
    announce("training step")
    rng = np.random.default_rng(12)
    n = 96
    x, dy = rng.standard_normal((200, n)), rng.standard_normal((200, n))
    gamma, beta = 1 + 0.1 * rng.standard_normal(n), 0.1 * rng.standard_normal(n)
    w, b = rng.standard_normal((n, n)) / np.sqrt(n), rng.standard_normal(n)
    args = [to_dev(v) for v in (x, dy, gamma, beta, w, b)]
    got = train_step(*args)
    y, mean, rstd = layers.layernorm(x, gamma, beta)
    z = y @ w + b
    g = dy * layers.slope(z, "gelu")
    dx, dgamma, dbeta = layers.layernorm_backward(g @ w.T, x, gamma, mean, rstd)
    want = (layers.act(z, "gelu") + x, dx + dy, dgamma, dbeta, y.T @ g, g.sum(0))
    for a, e in zip(got, want):
        np.testing.assert_allclose(host(a), e, rtol=0, atol=1e-11 * max(1, np.abs(e).max()))
    # captured and replayed, with eager work between
    static = [a.clone() for a in args]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train_step(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = train_step(*static)
    for k in range(3):
        static[0].copy_(args[0] * (k + 1))
        graph.replay()
        eager = train_step(args[0] * (k + 1), *args[1:])
        torch.cuda.synchronize()
        for a, e in zip(out, eager):
            assert torch.equal(a, e)


def test_given_stream_and_workspace():
    """A stream argument, a workspace of exactly the queried size, one byte less refused."""
    announce("stream and workspace arguments")
    d = device()
    rng = np.random.default_rng(20)
    a, b = to_dev(rng.standard_normal((70, 90))), to_dev(rng.standard_normal((90, 50)))
    want = ozk.ozk_dgemm_epilogue(a, b, 14, act="gelu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ozk.ozk_dgemm_epilogue(a, b, 14, act="gelu", stream=s)
    x = torch.randn(33, 130, device=d)
    s.wait_stream(torch.cuda.current_stream())
    y = ozk.ozk_layernorm(x, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(y, ozk.ozk_layernorm(x))
    need = ozk.ozk_dgemm_epilogue_grad_workspace_size(70, 50, 90, 14)
    dc = to_dev(rng.standard_normal((70, 50)))
    for size in (need, need - 1):
        ws = torch.empty(size, dtype=torch.uint8, device=d)
        if size == need:
            ozk.ozk_dgemm_epilogue_grad(dc, a, b, 14, workspace=ws)
        else:
            with pytest.raises(ozk.OzkError) as e:
                ozk.ozk_dgemm_epilogue_grad(dc, a, b, 14, workspace=ws)
            assert e.value.status == -2


def test_binding_refusals():
    """Shapes, types, strides and devices the binding refuses before any call."""
    announce("binding refusals")
    d = device()
    a = torch.zeros(4, 6, dtype=torch.float64, device=d)
    b = torch.zeros(6, 5, dtype=torch.float64, device=d)
    q = torch.zeros(4, 6, dtype=torch.int8, device=d)
    s = torch.zeros(4, device=d)
    for bad in (dict(b=b[:5]), dict(bias=b[0, :4]), dict(residual=a), dict(out=a), dict(preact=a),
                dict(residual=torch.zeros(5, dtype=torch.float64, device=d).expand(4, 5)),
                dict(act="swish"), dict(workspace=torch.zeros(8, device=d, dtype=torch.uint8)[::2])):
        with pytest.raises(ValueError):
            ozk.ozk_dgemm_epilogue(**dict(dict(a=a, b=b, r=14), **bad))
    with pytest.raises(ValueError):
        ozk.ozk_dgemm_epilogue(a[:, :1].expand(4, 6), b, 14)
    with pytest.raises(ValueError):
        ozk.ozk_dgemm_epilogue(b.t(), b, 14)
    with pytest.raises(TypeError):
        ozk.ozk_dgemm_epilogue(a, b, 14, bias=torch.zeros(5, device=d))
    with pytest.raises(TypeError):
        ozk.ozk_dgemm_epilogue(a, b, 14, bias=torch.zeros(5, dtype=torch.float64))
    with pytest.raises(ValueError):
        ozk.ozk_dgemm_epilogue_grad(torch.zeros(4, 5, dtype=torch.float64, device=d), a, b, 14,
                                    act="gelu")
    for bad in (dict(scale_x=s[:3]), dict(scale_w=s[:3]), dict(w=q[:, :5]), dict(residual=q.bfloat16()[:, :3]),
                dict(x=q[:1].expand(4, 6))):
        with pytest.raises(ValueError):
            ozk.ozk_int8linear(**dict(dict(x=q, scale_x=s, w=q, scale_w=s), **bad))
    with pytest.raises(TypeError):
        ozk.ozk_int8linear(q, s, q, s, bias=s)              # bf16 is asked for
    with pytest.raises(TypeError):
        ozk.ozk_int8linear(q, s, q, s, dtype=torch.float64)
    x = torch.zeros(4, 6, device=d)
    for f in (ozk.ozk_layernorm, lambda x, g: ozk.ozk_int8quant_rows(x, norm=True, gamma=g)):
        with pytest.raises(ValueError):
            f(x, s)
        with pytest.raises(TypeError):
            f(x, torch.zeros(6, device=d, dtype=torch.float64))
        with pytest.raises(ValueError):
            f(x.t(), s)
    with pytest.raises(ozk.OzkError):
        ozk.ozk_layernorm(x, eps=-1.0)
    with pytest.raises(ozk.OzkError):
        ozk.ozk_int8quant_rows(x, gamma=torch.zeros(6, device=d))   # weights without the norm
    with pytest.raises(TypeError):
        ozk.ozk_layernorm_backward(x, x, None, s.double(), s)
