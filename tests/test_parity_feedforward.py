"""GPU parity of the feed-forward operators against their plain 64-bit forms.

Tolerances count roundings, as in the layer operators' tests: u = 2^-24 (2^-53) is half a step
of the fp32 (fp64) arithmetic, eps / 2 of the output's type one rounding to it."""
import threading

import numpy as np
import pytest
import torch

import fp64_gemm_emulation_ozk_amd as ozk
import ozk_inputs
from oracle import feedforward as ff
from oracle import layers
from oracle import rns

import mx_plan
from gpu_common import announce, device, to_dev
from test_parity_layers import (TYPES, U32, U64, act_error, assert_near, half_step, host, padded,
                                tiny)

pytestmark = pytest.mark.gpu

SHORT = {k: v for k, v in TYPES.items() if k != "float64"}


# ------------------------------------------------------------------ codes
def matrix(rows, cols, dtype, seed):
    """Values of many sizes: blocks of their own scale, zeros, midpoints between codes."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-6, 7, (rows, cols)))
    x[rng.random((rows, cols)) < 0.1] = 0
    mids = np.array([0.25, -0.75, 1.25, -1.75, 2.5, 3.5, -5.0, 7.0, 4.0, -0.0])
    at = rng.random((rows, cols)) < 0.3
    x[at] = rng.choice(mids, int(at.sum()))
    return torch.from_numpy(x).to(dtype)


def byte_buffer(lines, width, pad, fill):
    buf = torch.full((lines + 1, width + pad), fill, dtype=torch.uint8, device=device())
    return buf, buf[:lines, :width]


def check_quant(x, axis, pad=0, offset=0):
    """Codes and scales bit for bit; nothing written beside them."""
    lines = host(x) if axis == 0 else host(x).T
    want, scales = ff.mx_quant(lines)
    n, k = lines.shape
    qb, q = byte_buffer(n, want.shape[1] // 2, 16 * pad, 77)
    sb, s = byte_buffer(n, want.shape[1] // 32, 8 * pad, 78)
    got = ozk.ozk_mxfp4_quant(padded(x, pad, offset), axis, codes=q, scales=s)
    assert got[0] is q and got[1] is s
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    np.testing.assert_array_equal(ff.mx_unpack(q.cpu().numpy()), want)
    assert (qb[n:] == 77).all() and (qb[:, q.shape[1]:] == 77).all()
    assert (sb[n:] == 78).all() and (sb[:, s.shape[1]:] == 78).all()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("axis", [0, 1])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 33), (33, 1), (5, 256), (256, 5), (7, 257),
                                       (257, 7), (64, 64), (129, 130), (300, 1000), (1000, 300),
                                       (3, 8192), (8192, 3), (513, 2049)])
def test_quant(kind, axis, rows, cols):
    announce(f"mxfp4 quant {kind} axis={axis} {rows} x {cols}")
    x = matrix(rows, cols, TYPES[kind], rows * 7 + cols)
    check_quant(x, axis)
    check_quant(x, axis, pad=3, offset=1)


@pytest.mark.parametrize("kind", ["float16", "bfloat16"])
def test_quant_every_value(kind):
    """Every bit pattern of the 16-bit types, in blocks of neighbours (each of one exponent or
    nearly so) and in blocks beside values 2^1 .. 2^5 times as large."""
    announce(f"mxfp4 quant every {kind}")
    bits = np.arange(65536, dtype=np.uint16).view(np.int16)
    v = torch.from_numpy(bits.copy()).view(TYPES[kind])
    x = v.view(256, 256).clone()
    check_quant(x, 0)
    check_quant(x.t().contiguous(), 1)
    finite = torch.where(torch.isfinite(v), v, torch.zeros_like(v)).view(-1, 16)
    for up in range(1, 6):
        big = (finite.abs().amax(1, keepdim=True).double() * 2.0 ** up).to(v.dtype)
        both = torch.cat((finite, big.expand(-1, 16)), 1).reshape(64, -1)
        check_quant(both, 0)
        check_quant(both, 1)


@pytest.mark.parametrize("axis", [0, 1])
def test_quant_doubles_next_to_midpoints(axis):
    """fp64 values one step to either side of a border between two codes."""
    announce("mxfp4 quant fp64 borders")
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    v = np.concatenate((mids, np.nextafter(mids, 0), np.nextafter(mids, 9), [6.0, 7.99, 4.0]))
    x = np.resize(np.concatenate((v, -v, [2.0 ** -60, -2.0 ** -1074])), (40, 64))
    x[:, ::32] = 4.0
    x = x * np.exp2(np.arange(-20, 20) * 5.0)[:, None]
    x = x if axis == 0 else x.T
    check_quant(torch.from_numpy(np.ascontiguousarray(x)), axis)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("axis", [0, 1])
def test_quant_edges(kind, axis):
    """Inf and NaN, the types' largest and smallest values, exponents past a scale's range."""
    announce(f"mxfp4 quant edges {kind} axis={axis}")
    dtype = TYPES[kind]
    fi = torch.finfo(dtype)
    x = torch.ones(12, 96, dtype=dtype)
    x[0, 3], x[1, 40], x[2, 70] = float("inf"), float("nan"), -float("inf")
    x[3] = fi.max
    x[4] = -fi.tiny
    x[5] = fi.tiny * fi.eps
    x[6] = 0
    x[7] = -0.0
    x[8, 32:64] = fi.tiny * 3
    x[9, 0] = fi.max
    if kind == "float64":
        x[3], x[9, 0], x[10] = 2.0 ** 130, 1.999 * 2.0 ** 129, 1e300
        x[11] = 2.0 ** -127
    check_quant(x if axis == 0 else x.t().contiguous(), axis)


def test_quant_empty():
    announce("mxfp4 quant empty")
    e = torch.empty(0, 70, device=device())
    q, s = ozk.ozk_mxfp4_quant(e)
    assert q.shape == (0, 128) and s.shape == (0, 8)
    q, s = ozk.ozk_mxfp4_quant(torch.empty(70, 0, device=device()), 1)
    assert q.shape == (0, 128) and s.shape == (0, 8)
    assert ozk.ozk_mxfp4_values(q, s, 70).shape == (0, 70)


def test_quant_many_lines():
    """Lines of several launches, and past 32-bit offsets: the same bytes as those lines alone."""
    announce("mxfp4 quant many lines")
    block = matrix(1021, 3, torch.bfloat16, 5).to(device())
    rows = 1021 * 135000   # past 2^27 lines of one step
    x = block.repeat(rows // 1021, 1)
    q, s = ozk.ozk_mxfp4_quant(x)
    wq, ws = ozk.ozk_mxfp4_quant(block)
    assert torch.equal(s.view(-1, 1021, 8), ws[None].expand(rows // 1021, -1, -1))
    for part in q.view(-1, 1021, 128).split(20000):
        assert torch.equal(part, wq[None].expand(len(part), -1, -1))
    del x
    v = ozk.ozk_mxfp4_values(q, s, 3, dtype=torch.bfloat16)
    wv = ozk.ozk_mxfp4_values(wq, ws, 3, dtype=torch.bfloat16)
    assert torch.equal(v.view(-1, 1021, 3), wv[None].expand(rows // 1021, -1, -1))


@pytest.mark.parametrize("kind,cols", [("bfloat16", (1 << 29) + 1), ("float64", (1 << 28) + 70)])
def test_quant_many_columns(kind, cols):
    """Columns of several launches, the last one of a single column."""
    announce(f"mxfp4 quant many columns {kind}")
    if torch.cuda.mem_get_info()[0] < cols * 160:
        pytest.skip("needs 160 bytes of device memory a column")
    block = matrix(1, 1021, TYPES[kind], 6).to(device())
    x = block.repeat(1, cols // 1021 + 1)[:, :cols]
    q, s = ozk.ozk_mxfp4_quant(x, 1)
    wq, ws = ozk.ozk_mxfp4_quant(block, 1)
    whole = cols // 1021 * 1021
    for got, want in ((q, wq), (s, ws)):
        for part in got[:whole].view(-1, 1021, got.shape[1]).split(20000):
            assert torch.equal(part, want[None].expand(len(part), -1, -1))
        assert torch.equal(got[whole:], want[:cols - whole])


@pytest.mark.parametrize("kind", list(TYPES))
def test_values_every_code_and_scale(kind):
    """All 16 codes under all 256 scales, rounded once to the type (fp16 overflows to Inf)."""
    announce(f"mxfp4 values {kind}")
    codes = np.tile(np.arange(16, dtype=np.uint8), (32, 16))
    scales = np.arange(256, dtype=np.uint8).reshape(32, 8)
    want = torch.from_numpy(ff.mx_values(codes, scales)).to(TYPES[kind])
    for k in (256, 255, 1, 37):
        out = torch.full((32, k + 3), 5.0, dtype=TYPES[kind], device=device())
        got = ozk.ozk_mxfp4_values(to_dev(ff.mx_pack(codes)), to_dev(scales), k, out=out[:, :k])
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=123.0),
                           torch.nan_to_num(want[:, :k], nan=123.0))
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want[:, :k]))
        assert (out[:, k:] == 5.0).all()


@pytest.mark.parametrize("lines,k", [(1, 1), (3, 300), (70, 256), (129, 1111), (2, 9000)])
def test_values(lines, k):
    announce(f"mxfp4 values {lines} x {k}")
    x = matrix(lines, k, torch.float32, k).to(device())
    q, s = ozk.ozk_mxfp4_quant(x)
    codes, scales = ff.mx_quant(host(x))
    for kind, dtype in TYPES.items():
        v = ozk.ozk_mxfp4_values(q, s, k, dtype=dtype)
        np.testing.assert_array_equal(host(v), ff.mx_values(codes, scales)[:, :k])


# ------------------------------------------------------------------ products on codes
def mx_operand(rng, lines, k, spread=2):
    """Random codes and scales near 2^0: (packed, scales, values)."""
    kp = ff.padded_k(k)
    codes = rng.integers(0, 16, (lines, kp)).astype(np.uint8)
    codes[:, k:] = 0
    scales = rng.integers(127 - spread, 128 + spread, (lines, kp // 32)).astype(np.uint8)
    return ff.mx_pack(codes), scales, ff.mx_values(codes, scales)[:, :k]


def line_pad(b, pad):
    """Lines as a view of a wider buffer, whose other bytes would spoil what reads them."""
    buf = torch.full((b.shape[0], b.shape[1] + pad), 255, dtype=torch.uint8, device=device())
    buf[:, :b.shape[1]] = to_dev(b)
    return buf[:, :b.shape[1]]


# one row to several tiles of rows; columns and K around the tiles, odd and ragged; K of one
# value, below a step, and long
LINEAR = [(1, 1, 1), (1, 16, 64), (1, 700, 1000), (2, 33, 129), (7, 4100, 257), (8, 130, 513),
          (9, 64, 2048), (16, 256, 4096), (17, 130, 1001), (31, 65, 128), (33, 1000, 300),
          (48, 272, 2048), (64, 128, 256), (65, 129, 256), (100, 515, 383), (128, 256, 512),
          (130, 300, 1024), (200, 96, 5000), (256, 256, 256), (300, 520, 384), (513, 257, 640),
          (1000, 1030, 130), (3, 48, 30000), (20, 100, 40000), (128, 128, 16384),
          (700, 2050, 1024),
          # enough tiles of 256 x 256 for every compute unit, several rounds of smaller ones
          (3000, 4500, 272), (2900, 4600, 700)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,n,k", LINEAR)
def test_product_is_exact(m, n, k, gated):
    """Sums that fp32 holds exactly, so that every order gives the same bits: products are
    multiples of 2^-4 and at most 36 * 2^2 (scales 2^-1 .. 2^1, or all 1 for long K), K sums of
    them below 2^24 steps."""
    announce(f"mxfp4 exact m={m} n={n} k={k} gated={gated}")
    rng = np.random.default_rng(m + n + k)
    spread = 1 if k <= 7000 else 0
    wide = 2 * n if gated else n
    xq, xs, xv = mx_operand(rng, m, k, spread)
    wq, ws, wv = mx_operand(rng, wide, k, spread)
    if spread == 0:
        assert (xs == 127).all()
    # fp64 sums of these are exact, on the GPU as well
    z = host(torch.matmul(to_dev(xv), to_dev(np.ascontiguousarray(wv.T))))
    for pad in (0, 1):
        args = (line_pad(xq, 16 * pad), line_pad(xs, 8 * pad), line_pad(wq, 32 * pad),
                line_pad(ws, 16 * pad))
        out = torch.full((m, n + pad), 7.0, device=device())
        if gated:
            ozk.ozk_mxfp4_gated(*args, act="none", out=out[:, :n])
            want = (z[:, :n].astype(np.float32) * z[:, n:].astype(np.float32)).astype(np.float64)
        else:
            ozk.ozk_mxfp4_linear(*args, out=out[:, :n])
            want = z
        np.testing.assert_array_equal(host(out[:, :n]), want)
        assert (out[:, n:] == 7.0).all()


def check_mx(got, xv, wv, bias, name, res, gated):
    """z: a sum of k products, each exact in fp32: at most 128 additions within an instruction,
    k / 128 from one to the next, 40 between waves and parts of a split K, each off by a step
    (2 u: the matrix cores may cut off) of the magnitudes' sum; then the bias.  An activation
    stretches an error by at most 1.13 and adds 16 roundings of |z|; the gate's product adds its own
    rounding and both factors' errors."""
    k = xv.shape[1]
    # the magnitudes' sum in 64 bits on the GPU: only its size matters
    z = host(torch.matmul(to_dev(xv), to_dev(np.ascontiguousarray(wv.T))))
    mag = host(torch.matmul(to_dev(np.abs(xv)), to_dev(np.ascontiguousarray(np.abs(wv).T))))
    ez = (168 + k / 128) * 2 * U32 * mag
    if bias is not None:
        z = z + host(bias)
        ez = ez + U32 * (np.abs(z) + ez)
    n = z.shape[1] // 2 if gated else z.shape[1]
    y = layers.act(z[:, :n], name)
    err = 1.13 * ez[:, :n] * 1.01 + (16 * U32 * np.abs(z[:, :n]) if name not in ("none", "relu")
                                     else 0)
    want = y
    if gated:
        up, eu = z[:, n:], ez[:, n:]
        want = y * up
        err = np.abs(y) * eu + np.abs(up) * err + err * eu + 2 * U32 * np.abs(want)
    elif res is not None:
        want = y + host(res)
        err = err + U32 * np.abs(want)
    assert_near(host(got), want, err + half_step(got.dtype) * (np.abs(want) + err)
                + tiny(got.dtype), f"mxfp4 {name} gated={gated}")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", list(SHORT))
@pytest.mark.parametrize("m,n,k", LINEAR)
def test_product(m, n, k, kind, gated):
    announce(f"mxfp4 product m={m} n={n} k={k} {kind} gated={gated}")
    rng = np.random.default_rng(m * n + k)
    dtype = TYPES[kind]
    wide = 2 * n if gated else n
    xq, xs, xv = mx_operand(rng, m, k)
    wq, ws, wv = mx_operand(rng, wide, k)
    # outputs of order 1: W's scales carry k^(-1/2) and the codes' size
    down = int(np.rint(np.log2(8 * np.sqrt(k))))
    ws, wv = (ws - down).astype(np.uint8), wv * 2.0 ** -down
    bias = torch.from_numpy(rng.standard_normal(wide)).to(dtype).to(device())
    res = torch.from_numpy(rng.standard_normal((m, n))).to(dtype).to(device())
    args = [to_dev(t) for t in (xq, xs, wq, ws)]
    pad = (m + n) % 3
    names = layers.ACTS if m * n < 10000 else layers.ACTS[(m + n + k) % 5:][:1] + ("none",)
    for name in names:
        out = torch.full((m, n + pad), 7.0, dtype=dtype, device=device())[:, :n]
        if gated:
            got = ozk.ozk_mxfp4_gated(*args, bias=bias, act=name, out=out)
            check_mx(got, xv, wv, bias, name, None, True)
            continue
        got = ozk.ozk_mxfp4_linear(*args, bias=bias, act=name, residual=res, out=out)
        check_mx(got, xv, wv, bias, name, res, False)
        over = res.clone()
        again = ozk.ozk_mxfp4_linear(*args, bias=bias, act=name, residual=over, out=over)
        assert torch.equal(again, got)
    plain = (ozk.ozk_mxfp4_gated(*args, act="silu", dtype=dtype) if gated else
             ozk.ozk_mxfp4_linear(*args, dtype=dtype))
    check_mx(plain, xv, wv, None, "silu" if gated else "none", None, gated)


def mx_operand_on_gpu(gen, lines, k):
    """As mx_operand with scales 2^-1 .. 2^1, a block's of its own: (packed, scales, values)."""
    kp = ff.padded_k(k)
    draw = lambda *a: torch.randint(*a, generator=gen, device=device())
    codes = draw(0, 16, (lines, kp))
    codes[:, k:] = 0
    scales = draw(126, 129, (lines, kp // 32))
    grid = torch.from_numpy(np.concatenate((ff.GRID, -ff.GRID))).to(device())
    values = grid[codes].view(lines, -1, 32) * torch.exp2((scales - 127).double())[:, :, None]
    codes = codes.to(torch.uint8)
    return codes[:, 0::2] | codes[:, 1::2] << 4, scales.to(torch.uint8), values.view(lines, kp)


def check_mx_exact(m, n, k, gated):
    """fp32 sums that are exact in every order, since the magnitudes of their terms, multiples of
    2^-4, sum to less than 2^20; then fp32 steps, the same here, and one rounding to the type.  The
    last step before fp16 may be one instruction with the rounding, which then rounds the exact
    product or sum once; by way of fp32 it is off by 2^-24 and by 2^-11 of what that gives (below
    fp16's normal range by 2^-25)."""
    gen = torch.Generator(device()).manual_seed(m * n + k)
    wide = 2 * n if gated else n
    xq, xs, xv = mx_operand_on_gpu(gen, m, k)
    wq, ws, wv = mx_operand_on_gpu(gen, wide, k)
    wt = wv.t().contiguous()
    assert torch.matmul(xv.abs(), wt.abs()).amax() < 2.0 ** 20
    z = torch.matmul(xv, wt).float()
    f = ozk.ozk_mxfp4_gated if gated else ozk.ozk_mxfp4_linear
    args = (xq, xs, wq, ws)
    want = z[:, :n] * z[:, n:] if gated else z
    for _ in range(2):
        out = torch.full((m, n + 3), 7.0, device=device())
        f(*args, act="none", out=out[:, :n])
        assert torch.equal(out[:, :n], want) and (out[:, n:] == 7.0).all()
    for dtype in SHORT.values():
        normal = lambda *s: torch.randn(s, generator=gen, device=device()).to(dtype)
        bias, res = normal(wide), normal(m, n)
        zb = z + bias.float()
        y, last = zb[:, :n].relu(), zb[:, n:] if gated else res.float()
        join = torch.mul if gated else torch.add
        kw = {} if gated else dict(residual=res)
        got = f(*args, bias=bias, act="relu", dtype=dtype, **kw)
        same = got == join(y, last).to(dtype)
        if dtype is torch.float16:
            exact = join(y.double(), last.double())
            same |= ((got.double() - exact).abs()
                     <= (2.0 ** -11 * (1 + 2.0 ** -24) + 2.0 ** -24) * exact.abs() + 2.0 ** -25)
        assert same.all()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,n,k", mx_plan.TILES)
def test_product_through_the_tiles_rings(m, n, k, gated):
    """Every tile, K whole and split, over many turns of its rings."""
    announce(f"mxfp4 tiles m={m} n={n} k={k} gated={gated} {mx_plan.plan(m, n, k, gated)}")
    check_mx_exact(m, n, k, gated)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,n,k", mx_plan.STREAM)
def test_product_through_the_streams_rings(m, n, k, gated):
    """Few rows: each number of rows and columns a workgroup takes."""
    announce(f"mxfp4 stream m={m} n={n} k={k} gated={gated} {mx_plan.plan(m, n, k, gated)}")
    check_mx_exact(m, n, k, gated)


@pytest.mark.parametrize("m", [1, 12, 40, 100, 300])
@pytest.mark.parametrize("gated", [False, True])
def test_product_of_every_scale(m, gated):
    """One block of a row against one block of a column under every pair of scales whose
    product fp32 holds; scales 255 give NaN in the outputs they touch and nowhere else."""
    announce(f"mxfp4 every scale m={m} gated={gated}")
    rng = np.random.default_rng(m)
    n, k = 256, 512
    for turn in range(4):
        xs = np.full((m, 16), 127, dtype=np.uint8)
        ws = np.full((2 * n if gated else n, 16), 127, dtype=np.uint8)
        codes = np.zeros((m, k), dtype=np.uint8)
        wcodes = np.zeros((ws.shape[0], k), dtype=np.uint8)
        block = 3 + 4 * turn      # another lane quarter, another half of a step
        codes[:, 32 * block + turn] = rng.integers(1, 8, m)
        wcodes[:, 32 * block + turn] = 8 + rng.integers(1, 8, ws.shape[0])
        xs[:, block] = rng.integers(1, 255, m)
        ws[:, block] = np.resize(np.arange(256), ws.shape[0])
        xv, wv = ff.mx_values(codes, xs), ff.mx_values(wcodes, ws)
        args = [to_dev(t) for t in (ff.mx_pack(codes), xs, ff.mx_pack(wcodes), ws)]
        with np.errstate(invalid="ignore", over="ignore"):
            z = xv[:, [32 * block + turn]] * wv[:, 32 * block + turn][None]
        if gated:
            # the gate alone: the other projection is 1
            wcodes[n:], ws[n:] = 0, 127
            one = np.concatenate((np.zeros(n), np.ones(n)))
            args[2], args[3] = to_dev(ff.mx_pack(wcodes)), to_dev(ws)
            got = host(ozk.ozk_mxfp4_gated(*args, act="none", dtype=torch.float32,
                                           bias=to_dev(one).float()))
            z = z[:, :n]
        else:
            got = host(ozk.ozk_mxfp4_linear(*args, dtype=torch.float32))
        np.testing.assert_array_equal(np.isnan(got), np.isnan(z))
        fits = (np.abs(z) < 2.0 ** 127) & (np.abs(z) >= 2.0 ** -126)
        np.testing.assert_array_equal(got[fits], z[fits])
        tiny_ones = np.abs(z) < 2.0 ** -126
        assert (np.abs(got[tiny_ones] - z[tiny_ones]) <= 2.0 ** -126).all()
        xs[:, block] = 255
        args[1] = to_dev(xs)
        if gated:
            assert torch.isnan(ozk.ozk_mxfp4_gated(*args)).all()
        else:
            assert torch.isnan(ozk.ozk_mxfp4_linear(*args)).all()


@pytest.mark.parametrize("m", [1, 20, 130])
def test_product_without_sums(m):
    """Empty operands; rows alone and among others; the longest K."""
    announce(f"mxfp4 edges m={m}")
    rng = np.random.default_rng(m)
    xq, xs, _ = mx_operand(rng, m, 700)
    wq, ws, _ = mx_operand(rng, 90, 700)
    x, sx, w, sw = [to_dev(t) for t in (xq, xs, wq, ws)]
    assert ozk.ozk_mxfp4_linear(x[:0], sx[:0], w, sw).shape == (0, 90)
    assert ozk.ozk_mxfp4_linear(x, sx, w[:0], sw[:0]).shape == (m, 0)
    assert ozk.ozk_mxfp4_gated(x[:0], sx[:0], w, sw).shape == (0, 45)
    # the longest K, constant: 131072 products of 9 / 4 are exact
    k = 131072
    codes = np.zeros((1, ff.padded_k(k)), dtype=np.uint8)
    codes[:, :k] = 3
    one = to_dev(ff.mx_pack(codes))
    sc = torch.full((1, one.shape[1] // 16), 127, dtype=torch.uint8, device=device())
    got = ozk.ozk_mxfp4_linear(one.expand(m, -1).contiguous(), sc.expand(m, -1).contiguous(),
                               one.expand(3, -1).contiguous(), sc.expand(3, -1).contiguous(),
                               dtype=torch.float32)
    assert (got == 131072 * 2.25).all()


@pytest.mark.parametrize("m", [3, 100])
def test_product_of_lines_of_fewer_values(m):
    """Operands of different k in as many steps: the shorter lines end in zeros.  Of different
    steps they are refused."""
    announce(f"mxfp4 lines of 300 and 400, m={m}")
    rng = np.random.default_rng(m)
    x, w = rng.integers(-3, 4, (m, 300)).astype(float), rng.integers(-3, 4, (70, 400)).astype(float)
    xq, wq = ozk.ozk_mxfp4_quant(to_dev(x)), ozk.ozk_mxfp4_quant(to_dev(w))
    want = x @ w[:, :300].T      # the values are codes times 2^-1 .. 2^0, and so are not rounded
    np.testing.assert_array_equal(host(ozk.ozk_mxfp4_values(*wq, 400)), w)
    np.testing.assert_array_equal(host(ozk.ozk_mxfp4_linear(*xq, *wq, dtype=torch.float32)), want)
    got = ozk.ozk_mxfp4_gated(*xq, *wq, act="none", dtype=torch.float32)
    np.testing.assert_array_equal(host(got), want[:, :35] * want[:, 35:])
    for f in (ozk.ozk_mxfp4_linear, ozk.ozk_mxfp4_gated):
        with pytest.raises(ValueError):
            f(*xq, *ozk.ozk_mxfp4_quant(to_dev(w[:, :256].copy())))


def test_product_far_rows():
    """C of more than 2^31 elements, and lines past 2^32 bytes."""
    announce("mxfp4 far rows")
    rng = np.random.default_rng(9)
    m, n, k = 70000, 33000, 256
    xq, xs, _ = mx_operand(rng, 1000, k)
    wq, ws, _ = mx_operand(rng, 1000, k)
    x, sx, w, sw = [to_dev(t) for t in (xq, xs, wq, ws)]
    want = ozk.ozk_mxfp4_linear(x, sx, w, sw)
    c = ozk.ozk_mxfp4_linear(x.repeat(70, 1), sx.repeat(70, 1), w.repeat(33, 1), sw.repeat(33, 1))
    assert c.shape == (m, n)
    for i in (0, 35, 69):
        for j in (0, 32):
            assert torch.equal(c[1000 * i:1000 * i + 1000, 1000 * j:1000 * j + 1000], want)
    del c
    # lines far apart: 300 lines of a leading dimension just below its bound
    far = torch.zeros(300 * ((1 << 24) - 16), dtype=torch.uint8, device=device())
    xf = far.as_strided((300, 128), ((1 << 24) - 16, 1))
    xf.copy_(x[:300])
    got = ozk.ozk_mxfp4_linear(xf, sx[:300], w, sw)
    assert torch.equal(got, want[:300])
    got = ozk.ozk_mxfp4_gated(x, sx, xf, sw[:300].contiguous())
    assert torch.equal(got, ozk.ozk_mxfp4_gated(x, sx, x[:300].contiguous(), sw[:300].contiguous()))


# ------------------------------------------------------------------ gated block in emulated fp64
@pytest.mark.parametrize("m,n,k,r,scaling", [(1, 1, 1, 14, "max"), (3, 31, 40, 14, "norm"),
                                             (64, 64, 64, 14, "max"), (70, 65, 129, 16, "norm"),
                                             (257, 33, 300, 18, "max"), (33, 150, 1000, 20, "max"),
                                             (300, 1000, 2100, 16, "norm"),
                                             (1100, 1025, 700, 15, "norm"), (2, 3000, 90, 2, "max"),
                                             (40, 127, 5000, 8, "norm")])
def test_dgemm_gated(m, n, k, r, scaling):
    """Z has the bits of ozk_dgemm_ex plus the bias; C is one product of the function's value."""
    announce(f"dgemm gated m={m} n={n} k={k} r={r} {scaling}")
    a, b = ozk_inputs.gemm_operands(m, 2 * n, k, seed=m + n + k, dist="phi", phi=0.5)
    bias = np.random.default_rng(m).standard_normal(2 * n)
    prod = host(ozk.ozk_dgemm_ex(to_dev(a), to_dev(b), r, scaling))
    for name, bi, pad in (("none", None, 0), ("relu", bias, 1), ("gelu", bias, 3),
                          ("gelu_tanh", None, 0), ("silu", bias, 2)):
        z = torch.full((m, 2 * n + pad), 5.0, dtype=torch.float64, device=device())
        c = torch.full((m, n + 2 * pad), 5.0, dtype=torch.float64, device=device())
        args = (padded(torch.from_numpy(a), pad), padded(torch.from_numpy(b), pad), r)
        kw = dict(bias=None if bi is None else to_dev(bi), act=name, scaling=scaling)
        ozk.ozk_dgemm_gated(*args, preact=z[:, :2 * n], out=c[:, :n], **kw)
        wz = prod if bi is None else prod + bi
        np.testing.assert_array_equal(host(z[:, :2 * n]), wz)
        y, up = layers.act(wz[:, :n], name), wz[:, n:]
        tol = (act_error(wz[:, :n], y) if name not in ("none", "relu") else 0 * y) * np.abs(up)
        # the product is rounded once here and once in the reference
        tol = tol * (1 + U64) + 2 * U64 * np.abs(y * up) * (tol > 0) + 2.0 ** -1074
        assert_near(host(c[:, :n]), y * up, tol, name)
        assert (z[:, 2 * n:] == 5.0).all() and (c[:, n:] == 5.0).all()
        assert torch.equal(ozk.ozk_dgemm_gated(*args, **kw), c[:, :n])   # Z not kept


@pytest.mark.parametrize("r", range(1, 21))
def test_dgemm_gated_every_r(r):
    """The reconstruction of both projections and of both gradients is compiled for every number
    of moduli: the bits of ozk_dgemm_ex.  Without an activation G is dC times the other half of Z,
    rounded once."""
    size = 300
    while rns.budget_q(r) - rns.ceil_log2(size) < 4:
        size //= 2
    m, n, k = size, max(size // 2, 1), max(size - 3, 1)
    announce(f"dgemm gated r={r} m={m} n={n} k={k}")
    a, b = [to_dev(x) for x in ozk_inputs.gemm_operands(m, 2 * n, k, seed=r, dist="phi", phi=1.0)]
    dc = to_dev(np.random.default_rng(r).standard_normal((m, n)))
    for scaling in ("max", "norm"):
        z = torch.empty((m, 2 * n), dtype=torch.float64, device=device())
        c = ozk.ozk_dgemm_gated(a, b, r, act="none", scaling=scaling, preact=z)
        assert torch.equal(z, ozk.ozk_dgemm_ex(a, b, r, scaling))
        assert torch.equal(c, z[:, :n] * z[:, n:])
        da, db, _ = ozk.ozk_dgemm_gated_grad(dc, a, b, r, z, act="none", scaling=scaling)
        g = torch.cat((dc * z[:, n:], dc * z[:, :n]), 1)
        assert torch.equal(da, ozk.ozk_dgemm_ex(g, b.t().contiguous(), r, scaling))
        assert torch.equal(db, ozk.ozk_dgemm_ex(a.t().contiguous(), g, r, scaling))


def test_dgemm_gated_edges():
    """Lines with Inf or NaN give NaN where they reach; no rows, no columns."""
    announce("dgemm gated edges")
    a, b = ozk_inputs.gemm_operands(40, 100, 70, seed=2, dist="phi", phi=1.0)
    a[7, 3], b[5, 11], b[6, 60] = np.nan, np.inf, np.nan
    c = host(ozk.ozk_dgemm_gated(to_dev(a), to_dev(b), 16, act="silu"))
    nan = np.isnan(c)
    assert nan[7].all() and nan[:, 11].all() and nan[:, 10].all()
    assert int(nan.sum()) == 50 + 2 * 39
    assert ozk.ozk_dgemm_gated(to_dev(a[:0]), to_dev(b), 14).shape == (0, 50)
    assert ozk.ozk_dgemm_gated(to_dev(a), to_dev(b)[:, :0], 14).shape == (40, 0)


@pytest.mark.parametrize("name", layers.ACTS)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (50, 35, 90), (300, 65, 64), (1025, 65, 20),
                                   (1500, 150, 33), (4200, 37, 9), (17, 300, 2100)])
def test_dgemm_gated_grad(m, n, k, name):
    """Against the formula in 64 bits.  G is off by 64 roundings (the slope's factors, the
    value's); a product's inner sums by that, by their own rounding in the reference, and by the
    scaled integers: half a unit of 2^-P of the line's maximum per term, P >= 44 for r = 16."""
    announce(f"dgemm gated grad {name} m={m} n={n} k={k}")
    rng = np.random.default_rng(m + n)
    a, b = rng.standard_normal((m, k)), rng.standard_normal((k, 2 * n))
    dc, z = rng.standard_normal((m, n)), 2 * rng.standard_normal((m, 2 * n))
    pad = m % 3
    da, db, dbias = ozk.ozk_dgemm_gated_grad(
        padded(torch.from_numpy(dc), pad), padded(torch.from_numpy(a), pad),
        padded(torch.from_numpy(b), pad), 16, padded(torch.from_numpy(z), pad), act=name)
    g = ff.gate_grad(dc, z, name)
    big = np.abs(z[:, :n])
    eg = 64 * U64 * np.concatenate((np.abs(dc * z[:, n:]) * (1 + big ** 2),
                                    np.abs(dc) * (1 + big)), axis=1)

    def tol(left, right, eleft, eright):
        inner = left.shape[1]
        scaled = inner * 2.0 ** -44 * np.abs(left).max(1)[:, None] * np.abs(right).max(0)
        return (eleft @ np.abs(right) + np.abs(left) @ eright
                + 2 * inner * U64 * (np.abs(left) @ np.abs(right)) + scaled)

    assert_near(host(da), g @ b.T, tol(g, b.T, eg, np.zeros_like(b.T)), "dA")
    assert_near(host(db), a.T @ g, tol(a.T, g, np.zeros_like(a.T), eg), "dB")
    assert_near(host(dbias), g.sum(0), eg.sum(0) + (m // 16 + 80) * U64 * np.abs(g).sum(0), "dbias")


def test_dgemm_gated_grad_is_the_difference_quotient():
    """The gradient of sum(dC * C) against central differences of the library's own forward: h =
    2^-16 leaves h^2 |f'''| / 6 (|f'''| below 1000 at these sizes: 4e-8) and 2^-52 |f| / h (|f| <
    1000: 1.5e-8)."""
    announce("dgemm gated grad differences")
    rng = np.random.default_rng(6)
    a, b, bias = rng.standard_normal((5, 4)), rng.standard_normal((4, 6)), rng.standard_normal(6)
    dc = rng.standard_normal((5, 3))
    z = torch.empty((5, 6), dtype=torch.float64, device=device())

    def f(a, b, bias):
        return float((dc * host(ozk.ozk_dgemm_gated(to_dev(a), to_dev(b), 20, act="gelu",
                                                    bias=to_dev(bias)))).sum())

    ozk.ozk_dgemm_gated(to_dev(a), to_dev(b), 20, act="gelu", bias=to_dev(bias), preact=z)
    grads = ozk.ozk_dgemm_gated_grad(to_dev(dc), to_dev(a), to_dev(b), 20, z, act="gelu")
    h = 2.0 ** -16
    for which, (v, g) in enumerate(zip((a, b, bias), grads)):
        for at in ((0,), (4,)) if v.ndim == 1 else ((0, 0), (3, 2), (1, 3)):
            e = np.zeros_like(v)
            e[at] = h
            up = [x + e if i == which else x for i, x in enumerate((a, b, bias))]
            dn = [x - e if i == which else x for i, x in enumerate((a, b, bias))]
            assert abs((f(*up) - f(*dn)) / (2 * h) - host(g)[at]) < 1e-7


def test_dgemm_gated_grad_parts():
    """Each gradient alone has the bits it has among all three; sums of no terms are zero."""
    announce("dgemm gated grad parts")
    rng = np.random.default_rng(4)
    a, b, dc, z = [to_dev(rng.standard_normal(s)) for s in ((40, 30), (30, 50), (40, 25),
                                                            (40, 50))]
    whole = ozk.ozk_dgemm_gated_grad(dc, a, b, 14, z)
    for i in range(3):
        need = dict(need_da=i == 0, need_db=i == 1, need_dbias=i == 2)
        part = ozk.ozk_dgemm_gated_grad(dc, a, b, 14, z, **need)
        assert [p is None for p in part] == [j != i for j in range(3)]
        assert torch.equal(part[i], whole[i])
    da, db, dbias = ozk.ozk_dgemm_gated_grad(dc[:0], a[:0], b, 14, z[:0])
    assert da.shape == (0, 30) and not db.any() and not dbias.any() and db.shape == (30, 50)
    wide = torch.full((40, 35), 2.0, dtype=torch.float64, device=device())
    da, db, dbias = ozk.ozk_dgemm_gated_grad(dc[:, :0], a, b[:, :0], 14, z[:, :0],
                                             da=wide[:, :30])
    assert not da.any() and (wide[:, 30:] == 2.0).all() and dbias.shape == (0,)


@pytest.mark.parametrize("m,n,k,r", [(1500, 1025, 1001, 16), (1344, 270, 1314, 16),
                                     (1997, 504, 303, 20), (640, 167, 1227, 8),
                                     (700, 700, 2000, 14), (2330, 716, 777, 14)])
def test_two_gradients_in_one_list_of_tiles(m, n, k, r):
    """Sizes whose two products are walked as one list of tiles, either of them the longer: the
    bits of each alone, in a workspace of the queried size and replayed from a graph."""
    announce(f"gradients in one list m={m} n={n} k={k} r={r}")
    rng = np.random.default_rng(m)
    a, b, dc, z = [to_dev(rng.standard_normal(s)) for s in ((m, k), (k, 2 * n), (m, n),
                                                            (m, 2 * n))]
    wide = torch.cat([dc, dc], 1)
    calls = [(lambda **kw: ozk.ozk_dgemm_gated_grad(dc, a, b, r, z, **kw),
              ozk.ozk_dgemm_gated_grad_workspace_size(m, n, k, r)),
             (lambda **kw: ozk.ozk_dgemm_epilogue_grad(wide, a, b, r, preact=z, act="silu", **kw),
              ozk.ozk_dgemm_epilogue_grad_workspace_size(m, 2 * n, k, r))]
    for f, need in calls:
        ws = torch.full((need + 1024,), 255, dtype=torch.uint8, device=device())
        whole = f(workspace=ws[:need])
        assert (ws[need:] == 255).all()
        da = f(need_db=False, need_dbias=False)[0]
        db = f(need_da=False, need_dbias=False)[1]
        assert torch.equal(whole[0], da) and torch.equal(whole[1], db)
        graph, out = captured(lambda: f(workspace=ws[:need]), [])
        for _ in range(3):
            for o in out:
                o.zero_()
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(o, w) for o, w in zip(out, whole))


@pytest.mark.parametrize("m,n,k,r,both_small", [(1500, 1025, 1001, 16, False),
                                                (1997, 504, 303, 20, True),
                                                (700, 700, 2000, 14, False)])
def test_gradients_in_the_larger_product_s_workspace(m, n, k, r, both_small):
    """Where the query counts both products' space, one that holds the larger alone gives the same
    bits, for both gradients and for either, and nothing past it is written; less is refused, and
    so is this much where both products are small (2^21 values in their operands at most).
    The products' own sizes are at least their planes and residues."""
    announce(f"gradients in less workspace m={m} n={n} k={k} r={r}")
    rng = np.random.default_rng(m)
    a, b, dc, z = [to_dev(rng.standard_normal(s)) for s in ((m, k), (k, 2 * n), (m, n),
                                                            (m, 2 * n))]
    wide = torch.cat([dc, dc], 1)
    up = lambda v, by: -(-v // by) * by
    least = lambda rows, cols, inner: r * up(inner, 128) * (rows + cols) + r * rows * up(cols, 64)
    one, two = sorted((least(m, k, 2 * n), least(k, 2 * n, m)))
    g = 16 * m * n
    calls = [(lambda **kw: ozk.ozk_dgemm_gated_grad(dc, a, b, r, z, **kw),
              ozk.ozk_dgemm_gated_grad_workspace_size(m, n, k, r)),
             (lambda **kw: ozk.ozk_dgemm_epilogue_grad(wide, a, b, r, preact=z, act="silu", **kw),
              ozk.ozk_dgemm_epilogue_grad_workspace_size(m, 2 * n, k, r))]
    for f, need in calls:
        assert need >= g + one + two                  # both are counted
        less = (need - one) // 256 * 256
        want = f()
        ws = torch.full((need,), 255, dtype=torch.uint8, device=device())
        if both_small:
            with pytest.raises(ozk.OzkError) as e:
                f(workspace=ws[:less])
            assert e.value.status == -2
            continue
        got = f(workspace=ws[:less])
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert (ws[less:] == 255).all()
        assert torch.equal(f(workspace=ws[:less], need_db=False, need_dbias=False)[0], want[0])
        assert torch.equal(f(workspace=ws[:less], need_da=False, need_dbias=False)[1], want[1])
        with pytest.raises(ozk.OzkError) as e:
            f(workspace=ws[:g + two - 256])
        assert e.value.status == -2


# ------------------------------------------------------------------ clipping
def clip_inputs(sizes, kinds, seed, size=1.0):
    rng = np.random.default_rng(seed)
    return [torch.from_numpy(rng.standard_normal(s) * size * 2.0 ** (i % 5)).to(TYPES[k])
            for i, (s, k) in enumerate(zip(sizes, kinds))]


def check_clip(norm, outs, xs, max_norm):
    """The norm: squares exact or rounded once in fp64, at most 2^20 additions in a row (2^8 here)
    between them, a root: 2^-44 relative.  An output: the factor's error, two roundings, one more
    to fp32 before a 16-bit type, and its type's."""
    want, clipped = ff.clip([host(x) for x in xs], max_norm)
    assert abs(float(norm) - want) <= 2.0 ** -44 * want
    for o, x, w in zip(outs, xs, clipped):
        assert o.dtype == x.dtype and o.shape == x.shape
        tol = (2.0 ** -43 + (U32 if o.element_size() == 2 else 0)) * np.abs(w)
        assert_near(host(o), w, tol + half_step(o.dtype) * (np.abs(w) + tol) + tiny(o.dtype),
                    "clipped")


@pytest.mark.parametrize("kind", list(TYPES) + ["all"])
@pytest.mark.parametrize("count", [1, 2, 7, 128, 129, 300])
def test_clip_norm(kind, count):
    """Tensors of 0 to many chunks, one launch and several, of one type and of all."""
    announce(f"clip {kind} {count} tensors")
    kinds = [k for k in TYPES] * count if kind == "all" else [kind] * count
    sizes = [(1, 16384, 0, 7, 4095, 16385, 100003, 33, 65536, 5000)[i % 10] for i in range(count)]
    xs = [x.to(device()) for x in clip_inputs(sizes, kinds[:count], count)]
    for max_norm in (1.0, 1e9, 0.0, float("inf")):
        keep = [x.clone() for x in xs]
        outs = [torch.full_like(x, 3.0) for x in xs]
        norm, got = ozk.ozk_clip_norm(xs, max_norm, out=outs)
        assert all(g is o for g, o in zip(got, outs))
        assert all(torch.equal(x, k) for x, k in zip(xs, keep))
        check_clip(norm, outs, xs, max_norm)
        again, same = ozk.ozk_clip_norm(keep, max_norm)     # in place
        assert torch.equal(again, norm)
        assert all(torch.equal(a, b) for a, b in zip(keep, outs))


def test_clip_norm_unaligned():
    """Tensors that start at any element, shapes of several dimensions, nothing written beside."""
    announce("clip unaligned")
    for kind, dtype in TYPES.items():
        buf = torch.full((200000,), 2.0, dtype=dtype, device=device())
        xs = [buf[1:1 + 40000].view(200, 200), buf[40003:40004], buf[50001:50001 + 131077]]
        keep = buf.clone()
        norm, outs = ozk.ozk_clip_norm(xs, 0.5)
        check_clip(norm, outs, [keep[1:40001].view(200, 200), keep[40003:40004],
                                keep[50001:181078]], 0.5)
        mask = torch.ones(200000, dtype=torch.bool, device=device())
        mask[1:40001] = mask[40003] = mask[50001:181078] = False
        assert torch.equal(buf[mask], keep[mask])


def test_clip_norm_of_other_orders():
    """Dense tensors whose dimensions lie in another order, as gradients of transposed weights: in
    place and into outputs of the same strides; outputs of others and gaps are refused."""
    announce("clip other orders")
    rng = np.random.default_rng(3)
    base = [to_dev(rng.standard_normal(s)).to(d) for s, d in (
        ((130, 70), torch.float32), ((3, 5, 7, 11), torch.bfloat16), ((6, 1, 9), torch.float64),
        ((257,), torch.float16))]
    views = [base[0].t(), base[1].permute(0, 3, 1, 2), base[2].permute(2, 1, 0), base[3]]
    assert not any(v.is_contiguous() for v in views[:3])
    norm, want = ozk.ozk_clip_norm(base, 1.0, out=[torch.empty_like(b) for b in base])
    outs = [torch.empty_like(v) for v in views]      # empty_like keeps the strides
    for o, v in zip(outs, views):
        assert o.stride() == v.stride()
    got, _ = ozk.ozk_clip_norm(views, 1.0, out=outs)
    assert torch.equal(got, norm)
    moved = [want[0].t(), want[1].permute(0, 3, 1, 2), want[2].permute(2, 1, 0), want[3]]
    assert all(torch.equal(o, w) for o, w in zip(outs, moved))
    for bad in (dict(tensors=views, out=[torch.empty_like(v).contiguous() for v in views]),
                dict(tensors=base[:1], out=[torch.empty(70, 130, device=device()).t()]),
                dict(tensors=[base[0][:, :69]]), dict(tensors=[base[0].t()[:69, ::2]]),
                dict(tensors=[base[0][:1].expand(4, 70)])):
        with pytest.raises(ValueError):
            ozk.ozk_clip_norm(**bad, max_norm=1.0)
    none = [base[0][:0].t(), torch.empty(70, 0, device=device())]   # empty: any strides
    ozk.ozk_clip_norm(views + none[:1], 1.0, out=outs + none[1:])
    assert all(torch.equal(o, w) for o, w in zip(outs, moved))
    ozk.ozk_clip_norm(views, 1.0)
    assert all(torch.equal(b, w) for b, w in zip(base, want))


def test_clip_norm_range():
    """Squares past fp64's range on either side; Inf and NaN leave the values as they are."""
    announce("clip range")
    for size in (1e-320, 1e-200, 1e-160, 1e-100, 1e100, 1e160, 1e200, 1e300):
        xs = [x.to(device()) for x in clip_inputs([40000, 3], ["float64"] * 2, 1, size)]
        outs = [torch.empty_like(x) for x in xs]
        norm, _ = ozk.ozk_clip_norm(xs, size, out=outs)
        want, clipped = ff.clip([host(x) for x in xs], size)
        assert abs(float(norm) - want) <= 2.0 ** -44 * want + 2.0 ** -1074
        for o, w in zip(outs, clipped):
            assert_near(host(o), w, 2.0 ** -43 * np.abs(w) + 2.0 ** -1073, "clipped")
    xs = [x.to(device()) for x in clip_inputs([40000, 3], ["float64"] * 2, 1, 1e307)]
    for x, bad in ((xs, None), ([xs[0].float()], np.inf),
                   ([torch.tensor([1.0, np.nan], device=device())], np.nan),
                   ([torch.tensor([1.0, -np.inf], device=device(), dtype=torch.float64)], np.inf)):
        outs = [torch.empty_like(t) for t in x]
        norm, _ = ozk.ozk_clip_norm(x, 1.0, out=outs)
        assert not np.isfinite(float(norm)) or bad is None
        if bad is None:   # the norm itself is past the range where the values are not
            continue
        keep = [t.clone() for t in x]
        ozk.ozk_clip_norm(x, 1.0)
        for o, t, k in zip(outs, x, keep):
            assert torch.equal(torch.nan_to_num(o, nan=7.0), torch.nan_to_num(k, nan=7.0))
            assert torch.equal(torch.nan_to_num(t, nan=7.0), torch.nan_to_num(k, nan=7.0))
    zero = [torch.zeros(5, device=device()), torch.zeros(0, device=device())]
    norm, outs = ozk.ozk_clip_norm(zero, 0.0)
    assert float(norm) == 0 and not outs[0].any()
    norm, outs = ozk.ozk_clip_norm(zero[1:], 1.0)
    assert float(norm) == 0


@pytest.mark.parametrize("size,max_norm", [(1e300, 1e-20), (1e300, 1e-30), (1e305, 1e-305),
                                           (1e300, 3e-8), (1e10, 1e-310), (1e305, 5e-324),
                                           (1e300, 0.0)])
def test_clip_norm_small_factor(size, max_norm):
    """Factors below fp64's normal range, down to none at all: the outputs are at most max_norm and
    as precise as where the factor is normal (test_clip_norm_range), to two steps of 2^-1074.  The
    values beside them in other types become 0."""
    announce(f"clip {size} to {max_norm}")
    xs = [x.to(device()) for x in clip_inputs([40000, 3], ["float64"] * 2, 7, size)]
    xs.append(torch.tensor([3e38, -1.0, 0.0], device=device()))
    xs.append(torch.tensor([6e4, -6e-8], dtype=torch.float16, device=device()))
    outs = [torch.full_like(x, 2.0) for x in xs]
    norm, _ = ozk.ozk_clip_norm(xs, max_norm, out=outs)
    # size is taken out of the values before squaring, and so of the factor
    units = [host(x) / size for x in xs]
    total = np.sqrt(sum((u * u).sum() for u in units))
    assert abs(float(norm) / size - total) <= 2.0 ** -43 * total
    for o, u in zip(outs[:2], units):
        want = u / total * max_norm
        assert_near(host(o), want, 2.0 ** -42 * np.abs(want) + 2.0 ** -1073, "clipped")
    assert not any(o.any() for o in outs[2:])
    keep = [x.clone() for x in xs]
    ozk.ozk_clip_norm(xs, max_norm)
    assert all(torch.equal(x, o) for x, o in zip(xs, outs)) and not torch.equal(keep[0], xs[0])


def test_clip_norm_large():
    """A tensor of more than 2^32 bytes and 2^31 elements among small ones."""
    announce("clip large")
    n = (1 << 31) + 12345
    x = torch.ones(n, dtype=torch.bfloat16, device=device())
    y = torch.full((100,), 2.0, device=device())
    norm, _ = ozk.ozk_clip_norm([y, x, y[:0]], 1.0)
    want = np.sqrt(n + 400.0)
    assert abs(float(norm) - want) <= 2.0 ** -44 * want
    assert torch.equal(x.amax(), x.amin())
    assert abs(float(x[-1]) - 1 / want) <= 2.0 ** -8 / want
    assert_near(host(y), np.full(100, 2 / want), 2.0 ** -23 * 2 / want, "y")


# ------------------------------------------------------------------ together
def serve(x, p, dtype):
    """A pre-norm gated feed-forward block on 4-bit codes:
    x + W2 (silu(Wg norm(x)) * Wu norm(x))."""
    y = ozk.ozk_layernorm(x, p["gamma"], p["beta"])
    h = ozk.ozk_mxfp4_gated(*ozk.ozk_mxfp4_quant(y), *p["w1"], bias=p["b1"], dtype=dtype)
    return ozk.ozk_mxfp4_linear(*ozk.ozk_mxfp4_quant(h), *p["w2"], bias=p["b2"], residual=x,
                                dtype=dtype)


def serve_weights(width, hidden, dtype, seed):
    rng = np.random.default_rng(seed)
    w = {"gamma": 1 + 0.1 * rng.standard_normal(width), "beta": 0.1 * rng.standard_normal(width),
         "b1": 0.1 * rng.standard_normal(2 * hidden), "b2": 0.1 * rng.standard_normal(width)}
    p = {k: torch.from_numpy(v).to(dtype).to(device()) for k, v in w.items()}
    for name, shape in (("w1", (2 * hidden, width)), ("w2", (width, hidden))):
        p[name] = ozk.ozk_mxfp4_quant(to_dev(rng.standard_normal(shape) / np.sqrt(shape[1])))
    return p


@pytest.mark.parametrize("tokens", [1, 9, 200])
def test_serving_block(tokens):
    """Step by step: each step's output against the plain form of that step on the step's own
    inputs, so that a code's rounding does not enter twice."""
    announce(f"mxfp4 block tokens={tokens}")
    dtype = torch.bfloat16
    p = serve_weights(264, 1040, dtype, 1)
    x = torch.from_numpy(np.random.default_rng(2).standard_normal((tokens, 264))).to(dtype)
    x = x.to(device())
    values = lambda q, s, k: ff.mx_values(ff.mx_unpack(q.cpu().numpy()), s.cpu().numpy())[:, :k]
    y = ozk.ozk_layernorm(x, p["gamma"], p["beta"])
    check_quant(y.cpu(), 0)
    yq = ozk.ozk_mxfp4_quant(y)
    h = ozk.ozk_mxfp4_gated(*yq, *p["w1"], bias=p["b1"], dtype=dtype)
    check_mx(h, values(*yq, 264), values(*p["w1"], 264), p["b1"], "silu", None, True)
    check_quant(h.cpu(), 0)
    hq = ozk.ozk_mxfp4_quant(h)
    out = serve(x, p, dtype)
    check_mx(out, values(*hq, 1040), values(*p["w2"], 1040), p["b2"], "none", x, False)


def captured(f, static):
    """f(*static) run once on a side stream, then captured: (graph, outputs)."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f(*static)
    return graph, out


@pytest.mark.parametrize("tokens", [5, 24, 150])
def test_serving_block_captured_and_on_streams(tokens):
    """Captured into a graph and replayed with new tokens between eager calls, and eager on two
    streams at once, the block gives the eager bits every time."""
    announce(f"mxfp4 block captured tokens={tokens}")
    dtype = torch.bfloat16
    p = serve_weights(2048, 1536, dtype, 3)
    rng = np.random.default_rng(4)
    batches = [torch.from_numpy(rng.standard_normal((tokens, 2048))).to(dtype).to(device())
               for _ in range(4)]
    want = [serve(x, p, dtype) for x in batches]
    static = batches[0].clone()
    graph, out = captured(lambda x: serve(x, p, dtype), [static])
    for turn in range(3):
        for x, y in zip(batches, want):
            static.copy_(x)
            graph.replay()
            assert torch.equal(serve(x, p, dtype), y)
            torch.cuda.synchronize()
            assert torch.equal(out, y)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            got.append(serve(batches[i % 4], p, dtype))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 4])


def train_step(x, dout, gamma, beta, w1, b1, w2, b2):
    """A pre-norm gated block in emulated fp64 with its input as residual, all gradients, and
    their clipping to norm 1 (in place)."""
    y, mean, rstd = ozk.ozk_layernorm(x, gamma, beta, stats=True)
    z = torch.empty((x.shape[0], w1.shape[1]), dtype=torch.float64, device=x.device)
    h = ozk.ozk_dgemm_gated(y, w1, 16, bias=b1, act="silu", scaling="norm", preact=z)
    out = ozk.ozk_dgemm_epilogue(h, w2, 16, bias=b2, residual=x, scaling="norm")
    dh, dw2, db2 = ozk.ozk_dgemm_epilogue_grad(dout, h, w2, 16, scaling="norm")
    dy, dw1, db1 = ozk.ozk_dgemm_gated_grad(dh, y, w1, 16, z, act="silu", scaling="norm")
    dx, dgamma, dbeta = ozk.ozk_layernorm_backward(dy, x, gamma, mean, rstd)
    norm, _ = ozk.ozk_clip_norm([dgamma, dbeta, dw1, db1, dw2, db2], 1.0)
    return out, dx + dout, norm, dgamma, dbeta, dw1, db1, dw2, db2


def test_training_step():
    """Against the same chain in 64 bits: a relative 1e-11 leaves room for the widths of the
    scaled integers (2^-44 of the line's maximum, inner sums of at most 256 terms)."""
    announce("gated training step")
    rng = np.random.default_rng(12)
    n, hid = 96, 128
    x, dout = rng.standard_normal((200, n)), rng.standard_normal((200, n))
    gamma, beta = 1 + 0.1 * rng.standard_normal(n), 0.1 * rng.standard_normal(n)
    w1, b1 = rng.standard_normal((n, 2 * hid)) / np.sqrt(n), rng.standard_normal(2 * hid)
    w2, b2 = rng.standard_normal((hid, n)) / np.sqrt(hid), rng.standard_normal(n)
    args = [to_dev(v) for v in (x, dout, gamma, beta, w1, b1, w2, b2)]
    got = train_step(*args)
    y, mean, rstd = layers.layernorm(x, gamma, beta)
    z = y @ w1 + b1
    h = ff.gate(z, "silu")
    dh = dout @ w2.T
    g = ff.gate_grad(dh, z, "silu")
    dx, dgamma, dbeta = layers.layernorm_backward(g @ w1.T, x, gamma, mean, rstd)
    norm, clipped = ff.clip([dgamma, dbeta, y.T @ g, g.sum(0), h.T @ dout, dout.sum(0)], 1.0)
    want = [h @ w2 + b2 + x, dx + dout, np.array(norm)] + clipped
    for a, e in zip(got, want):
        np.testing.assert_allclose(host(a), e, rtol=0, atol=1e-11 * max(1, np.abs(e).max()))
    # captured and replayed, with eager work between
    static = [a.clone() for a in args]
    graph, out = captured(train_step, static)
    for k in range(3):
        static[0].copy_(args[0] * (k + 1))
        graph.replay()
        eager = train_step(args[0] * (k + 1), *args[1:])
        torch.cuda.synchronize()
        for a, e in zip(out, eager):
            assert torch.equal(a, e)


def test_graphs_share_a_workspace():
    """Two graphs that were captured with one workspace, replayed in turn on one stream."""
    announce("feed-forward graphs with one workspace")
    rng = np.random.default_rng(31)
    a, b = to_dev(rng.standard_normal((70, 300))), to_dev(rng.standard_normal((300, 130)))
    x, w = [ozk.ozk_mxfp4_quant(to_dev(rng.standard_normal((s, 16384)))) for s in (90, 100)]
    grads = [to_dev(rng.standard_normal(s)) for s in (70000, 3)]
    ws = torch.empty(max(ozk.ozk_dgemm_gated_workspace_size(70, 65, 300, 14),
                         ozk.ozk_mxfp4_linear_workspace_size(90, 100, 16384),
                         ozk.ozk_clip_norm_workspace_size(2)), dtype=torch.uint8, device=device())
    kw = dict(workspace=ws)

    def first(a, b):
        outs = [torch.empty_like(g) for g in grads]
        norm, _ = ozk.ozk_clip_norm(grads, 1.0, out=outs, **kw)
        return ozk.ozk_dgemm_gated(a, b, 14, **kw), norm, *outs

    def second(*lines):
        return (ozk.ozk_mxfp4_linear(*lines, **kw),)

    graphs = [(captured(first, [a, b]), first(a, b)), (captured(second, [*x, *w]), second(*x, *w))]
    for turn in range(4):
        ws.fill_(255)
        for (graph, out), want in graphs:
            for o in out:
                o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(o, e) for o, e in zip(out, want))


def test_threads_on_streams_of_their_own():
    """Four host threads, each with a stream, run a serving block, a training step and a clipping
    at once: the bits of each alone."""
    announce("feed-forward threads")
    dtype = torch.bfloat16
    p = serve_weights(520, 700, dtype, 5)
    rng = np.random.default_rng(6)
    n, hid = 96, 128
    jobs = []
    for i in range(4):
        x = torch.from_numpy(rng.standard_normal((5 + 40 * i, 520))).to(dtype).to(device())
        args = [to_dev(rng.standard_normal(s)) for s in ((200, n), (200, n), (n,), (n,),
                                                         (n, 2 * hid), (2 * hid,), (hid, n), (n,))]
        jobs.append((x, args))
    want = [(serve(x, p, dtype), train_step(*args)) for x, args in jobs]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        x, args = jobs[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got[i] = (serve(x, p, dtype), train_step(*args))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0])
        assert all(torch.equal(a, b) for a, b in zip(g[1], w[1]))


def test_linear_gradients_on_codes():
    """The products of a linear layer's gradient on codes of both directions: dX = dC W with
    both along n, dW = dC^T X with both along m."""
    announce("mxfp4 gradients")
    m, n, k = 130, 75, 200
    rng = np.random.default_rng(8)
    dc, x, w = [torch.from_numpy(rng.standard_normal(s)).float().to(device())
                for s in ((m, n), (m, k), (n, k))]
    dx = ozk.ozk_mxfp4_linear(*ozk.ozk_mxfp4_quant(dc), *ozk.ozk_mxfp4_quant(w, 1),
                              dtype=torch.float32)
    dw = ozk.ozk_mxfp4_linear(*ozk.ozk_mxfp4_quant(dc, 1), *ozk.ozk_mxfp4_quant(x, 1),
                              dtype=torch.float32)
    val = lambda t: ff.mx_values(*ff.mx_quant(t))[:, :t.shape[1]]
    check_mx(dx, val(host(dc)), val(host(w).T), None, "none", None, False)
    check_mx(dw, val(host(dc).T), val(host(x).T), None, "none", None, False)


def test_given_stream_and_workspace():
    """A stream argument, a workspace of exactly the queried size, one byte less refused."""
    announce("feed-forward streams and workspaces")
    rng = np.random.default_rng(20)
    a, b, bias = [to_dev(rng.standard_normal(s)) for s in ((70, 90), (90, 100), (100,))]
    dc, z = to_dev(rng.standard_normal((70, 50))), to_dev(rng.standard_normal((70, 100)))
    xq, wq = ozk.ozk_mxfp4_quant(a), ozk.ozk_mxfp4_quant(b, 1)
    xl, wl = [to_dev(rng.standard_normal((s, 16384))) for s in (40, 100)]
    xlq, wlq = ozk.ozk_mxfp4_quant(xl), ozk.ozk_mxfp4_quant(wl)
    grads = [a.clone(), bias.float()]
    calls = [
        (lambda **kw: ozk.ozk_dgemm_gated(a, b, 14, bias=bias, **kw),
         ozk.ozk_dgemm_gated_workspace_size(70, 50, 90, 14)),
        (lambda **kw: ozk.ozk_dgemm_gated_grad(dc, a, b, 14, z, **kw),
         ozk.ozk_dgemm_gated_grad_workspace_size(70, 50, 90, 14)),
        (lambda **kw: ozk.ozk_mxfp4_linear(*xlq, *wlq, **kw),
         ozk.ozk_mxfp4_linear_workspace_size(40, 100, 16384)),
        (lambda **kw: ozk.ozk_mxfp4_gated(*xlq, *wlq, **kw),
         ozk.ozk_mxfp4_gated_workspace_size(40, 50, 16384)),
        (lambda **kw: ozk.ozk_clip_norm(grads, 0.5, out=[torch.empty_like(g) for g in grads],
                                        **kw)[1],
         ozk.ozk_clip_norm_workspace_size(2)),
        (lambda **kw: ozk.ozk_mxfp4_linear(*xq, *wq, **kw), None),
        (lambda **kw: ozk.ozk_mxfp4_quant(a, **kw), None),
        (lambda **kw: ozk.ozk_mxfp4_values(*xq, 90, **kw), None)]
    flat = lambda r: [r] if isinstance(r, torch.Tensor) else list(r)
    for f, need in calls:
        want = flat(f())
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = flat(f(stream=s))
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
        if need:
            ws = torch.full((need,), 255, dtype=torch.uint8, device=device())
            assert all(torch.equal(g, w) for g, w in zip(flat(f(workspace=ws)), want))
            with pytest.raises(ozk.OzkError) as e:
                f(workspace=torch.empty(need - 1, dtype=torch.uint8, device=device()))
            assert e.value.status == -2


def test_matrices_of_one_column():
    """Their column stride says nothing: a transposed row is as good as a column."""
    announce("one column of any stride")
    rng = np.random.default_rng(2)
    a, b = to_dev(rng.standard_normal((1, 40))).t(), to_dev(rng.standard_normal((1, 12)))
    assert a.shape == (40, 1) and a.stride(1) == 40
    dc, z = to_dev(rng.standard_normal((40, 6))), to_dev(rng.standard_normal((40, 12)))
    for f in (lambda a: ozk.ozk_dgemm_gated(a, b, 14),
              lambda a: ozk.ozk_dgemm_gated_grad(dc, a, b, 14, z)[1],
              lambda a: ozk.ozk_dgemm_ex(a, b, 14, "norm"),
              lambda a: ozk.ozk_mxfp4_quant(a)[0], lambda a: ozk.ozk_mxfp4_quant(a, 1)[1]):
        assert torch.equal(f(a), f(a.clone(memory_format=torch.contiguous_format).view(-1)[:, None]))


def test_rows_that_overlap_are_refused():
    """By every binding of a matrix: as leading dimension of an expanded row the library would take
    its length, and read past its end."""
    announce("rows that overlap")
    row = torch.zeros(1, 8, dtype=torch.float64, device=device())
    a, good = row.expand(8, 8), torch.zeros(8, 8, dtype=torch.float64, device=device())
    slid = torch.zeros(40, dtype=torch.float64, device=device()).unfold(0, 8, 4)[:8]
    i8 = torch.zeros(1, 8, dtype=torch.int8, device=device()).expand(8, 8)
    for bad in (a, slid, row[:, :1].expand(8, 1)):
        for f in (lambda t: ozk.ozk_dgemm(t, good[:t.shape[1]], 14),
                  lambda t: ozk.ozk_dgemm(good[:, :8], t, 14),
                  lambda t: ozk.ozk_dgemm_ex(t, good[:t.shape[1]], 14),
                  lambda t: ozk.ozk_dgemv(t, good[:t.shape[1], :2], 14),
                  lambda t: ozk.ozk_dgemv(good, t, 14), lambda t: ozk.ozk_deconstruct(t, 0, 14),
                  lambda t: ozk.ozk_dgemm_gated(t, good[:t.shape[1]], 14),
                  lambda t: ozk.ozk_mxfp4_quant(t), lambda t: ozk.ozk_layernorm(t)):
            with pytest.raises(ValueError):
                f(bad)
    for f in (ozk.ozk_int8gemm_fp4limb, ozk.ozk_int8gemm_fp4awe, ozk.ozk_int4int8gemm_fp4awe):
        with pytest.raises(ValueError):
            f(i8, i8.contiguous())
        with pytest.raises(ValueError):
            f(i8.contiguous(), i8)


def test_binding_refusals():
    """Shapes, types, strides and devices the binding refuses before any call."""
    announce("feed-forward binding refusals")
    d = device()
    a, b, z = [torch.zeros(s, dtype=torch.float64, device=d) for s in ((4, 6), (6, 10), (4, 10))]
    for bad in (dict(b=b[:5]), dict(b=b[:, :9]), dict(bias=b[0, :5]), dict(out=z), dict(preact=a),
                dict(act="swish"), dict(scaling="x"), dict(a=a[:, :1].expand(4, 6))):
        with pytest.raises(ValueError):
            ozk.ozk_dgemm_gated(**dict(dict(a=a, b=b, r=14), **bad))
    with pytest.raises(TypeError):
        ozk.ozk_dgemm_gated(a, b, 14, bias=torch.zeros(10, device=d))
    dc = torch.zeros(4, 5, dtype=torch.float64, device=d)
    for bad in (dict(preact=None), dict(preact=a), dict(b=b[:, :8]), dict(a=a[:3]), dict(da=b),
                dict(dbias=b[0, :5])):
        with pytest.raises(ValueError):
            ozk.ozk_dgemm_gated_grad(**dict(dict(dc=dc, a=a, b=b, r=14, preact=z), **bad))
    q, s = ozk.ozk_mxfp4_quant(torch.ones(6, 300, device=d))
    for f in (ozk.ozk_mxfp4_linear, ozk.ozk_mxfp4_gated):
        good = dict(x=q, scale_x=s, w=q, scale_w=s)
        for bad in (dict(scale_x=s[:5]), dict(scale_w=s[:, :8]), dict(x=q[:, :128]),
                    dict(w=q[:, :100]), dict(x=q[:, :0], scale_x=s[:, :0]), dict(scale_x=None),
                    dict(bias=torch.zeros(5, device=d, dtype=torch.bfloat16)),
                    dict(out=torch.zeros(6, 5, device=d)), dict(x=q[:1].expand(6, 256)),
                    dict(act="swish")):
            with pytest.raises(ValueError):
                f(**dict(good, **bad))
        with pytest.raises(TypeError):
            f(**dict(good, scale_x=s.to(torch.int8)))
        with pytest.raises(TypeError):
            f(**dict(good, bias=torch.zeros(6, device=d)))       # bf16 is asked for
        with pytest.raises(ozk.OzkError):                        # lines at an odd address
            buf = torch.zeros(6, 272, dtype=torch.uint8, device=d)
            f(**dict(good, x=buf[:, 8:264]))
    with pytest.raises(ValueError):
        ozk.ozk_mxfp4_gated(q[:5], s[:5], q[:5], s[:5])          # an odd number of lines
    for k in (512 + 1, 256, 0):
        with pytest.raises(ValueError):
            ozk.ozk_mxfp4_values(q, s, k)
    with pytest.raises(ValueError):
        ozk.ozk_mxfp4_quant(torch.ones(4, 4, device=d), 2)
    with pytest.raises(ValueError):
        ozk.ozk_mxfp4_quant(torch.ones(4, 8, device=d)[:, ::2])
    x = torch.ones(10, device=d)
    for bad in (dict(tensors=[x[::2]]), dict(tensors=[x], out=[x[:5]]),
                dict(tensors=[x], out=[x.double()]), dict(tensors=[x, x], out=[x]),
                dict(tensors=[x], norm=x)):
        with pytest.raises((ValueError, TypeError)):
            ozk.ozk_clip_norm(**dict(dict(max_norm=1.0), **bad))
    with pytest.raises(TypeError):
        ozk.ozk_clip_norm([x.int()], 1.0)
    for bad in ([x, x], [x, x[3:]]):                             # in place twice
        with pytest.raises(ozk.OzkError):
            ozk.ozk_clip_norm(bad, 1.0)
    with pytest.raises(ozk.OzkError):
        ozk.ozk_clip_norm([x], -1.0)
