"""The residual RMS norm, forward, in 8 bits and backward, on rows that no 16-byte access can take: slices of wider
rows at any offset and stride, tensors at any address of their type.  Tolerances as in the norm's own tests: the
same arithmetic, a row's terms spread over its threads in another order (at most 32 to a thread)."""
import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from oracle import layer as ol
from test_layer_gpu import BF16, DEV, F32, FP8, built, check_h, check_quantised, f64, rand, within  # noqa: F401

pytestmark = pytest.mark.gpu

# One row a half or whole warp, several a block, whole blocks, two and four chunks of eight a thread.
SIZES = [(5, 8), (3, 9), (70, 37), (2500, 96), (3, 129), (2440, 200), (4, 256), (7, 264), (2450, 505), (6, 1000), (5, 1001), (2433, 1032),
         (2, 4095), (3, 4104), (2, 8192), (3, 8200), (2, 16383), (2, 16384)]


def slice_of(shape, seed, dtype, off, pad, scale=1.5):
    """Values in rows `pad` wider, from the off-th value of the buffer on, NaN around them."""
    rows, D = shape
    flat = torch.full((rows * (D + pad) + off + 16,), float("nan"), dtype=dtype, device=DEV)
    t = flat[off:off + rows * (D + pad)].view(rows, D + pad)[:, :D]
    t.copy_(rand(shape, seed, scale, F32))
    return t


def at(shape, dtype, off):
    """A dense tensor from the off-th value of a buffer of sevens on, and the buffer."""
    n = torch.Size(shape).numel()
    flat = torch.full((n + off + 16,), 7.0, dtype=dtype, device=DEV)
    return flat[off:off + n].view(shape), flat


def untouched(flat, n, off):
    return bool((flat[:off] == 7).all() and (flat[off + n:] == 7).all())


# off and pad of x, of the stream, and the offsets of w, out and h
LIE = {
    "x at an odd place": ((1, 0), (0, 0), 0, 0, 0), "x in odd rows": ((0, 3), (0, 0), 0, 0, 0), "both in odd rows": ((3, 5), (1, 1), 0, 0, 0),
    "stream at an odd place": ((0, 0), (5, 0), 0, 0, 0), "stream in odd rows": ((0, 0), (0, 7), 0, 0, 0), "w": ((0, 0), (0, 0), 1, 0, 0),
    "out": ((0, 0), (0, 0), 0, 3, 0), "h": ((0, 8), (0, 0), 0, 0, 1), "all": ((1, 9), (3, 2), 3, 1, 5),
}


@pytest.mark.parametrize("rows,D", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lie", sorted(LIE))
def test_norm(rows, D, dtype, lie):
    (xo, xp), (ro, rp), wo, oo, ho = LIE[lie]
    x, r = slice_of((rows, D), 1, BF16, xo, xp), slice_of((rows, D), 2, dtype, ro, rp, 2.0)
    w, _ = at((D,), F32, wo)
    w.copy_(1 + rand((D,), 3, 0.2, F32))
    (out, o_flat), (h, h_flat) = at((rows, D), BF16, oo), at((rows, D), dtype, ho)
    pkg.add_rmsnorm(x, r, w, 1e-5, out=out, h=h)
    check_h(h, x, r)
    want = ol.rmsnorm(f64(h), f64(w), 1e-5)
    within(out, want, (2.0 ** -8 + 2.0 ** -17) * abs(want))
    assert untouched(o_flat, rows * D, oo) and untouched(h_flat, rows * D, ho)


@pytest.mark.parametrize("rows,D", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lie", ["x at an odd place", "both in odd rows", "w", "h", "all"])
def test_norm_in_8_bits(rows, D, dtype, lie):
    (xo, xp), (ro, rp), wo, _, ho = LIE[lie]
    x, r = slice_of((rows, D), 11, BF16, xo, xp), slice_of((rows, D), 12, dtype, ro, rp, 2.0)
    w, _ = at((D,), F32, wo)
    w.copy_(1 + rand((D,), 13, 0.2, F32))
    h, h_flat = at((rows, D), dtype, ho)
    row = (D + 15) // 16 * 16 + 16
    room = torch.full((rows + 1, row), 0x55, dtype=torch.uint8, device=DEV)
    q, s, _ = pkg.add_rmsnorm_fp8(x, r, w, 1e-5, out=room.view(FP8)[:rows, :D], h=h)
    check_h(h, x, r)
    check_quantised(q, s, ol.rmsnorm(f64(h), f64(w), 1e-5))
    assert (room[:rows, D:] == 0x55).all() and (room[rows] == 0x55).all() and untouched(h_flat, rows * D, ho)


@pytest.mark.parametrize("rows,D", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_without_residual(rows, D, dtype):
    """Of a slice at an odd place, bf16 and 8 bits."""
    x, w = slice_of((rows, D), 21, dtype, 1, 3), 1 + rand((D,), 22, 0.2, F32)
    want = ol.rmsnorm(f64(x), f64(w), 1e-5)
    out, h = pkg.add_rmsnorm(x, None, w, 1e-5)
    assert h is x
    within(out, want, (2.0 ** -8 + 2.0 ** -17) * abs(want))
    q, s, h = pkg.add_rmsnorm_fp8(x, None, w, 1e-5)
    assert h is x
    check_quantised(q, s, want)


@pytest.mark.parametrize("rows,D", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("odd", ["h", "w", "dout", "dh", "dx", "dresidual", "all", "without dh"])
def test_norm_backward(rows, D, dtype, odd):
    def place(name, shape, kind, seed=None, scale=1.0):
        off = 1 if odd in (name, "all", "without dh") else 0
        t, flat = at(shape, kind, off)
        if seed is not None:
            t.copy_(rand(shape, seed, scale, F32))
        return t, flat, off

    h, w = place("h", (rows, D), dtype, 31, 2.0)[0], place("w", (D,), F32, 32)[0]
    w += 1
    dout = place("dout", (rows, D), BF16, 33)[0]
    dh = None if odd == "without dh" else place("dh", (rows, D), dtype, 34)[0]
    dx, dr = place("dx", (rows, D), BF16), place("dresidual", (rows, D), dtype)
    g = pkg.add_rmsnorm_backward(h, w, dout, dh, 1e-5, grads=dict(dx=dx[0], dresidual=dr[0]))
    d, dw, size, wsize = ol.rmsnorm_backward(f64(h), f64(w), f64(dout), None if dh is None else f64(dh), 1e-5)
    within(g["dx"], d, 2.0 ** -8 * abs(d) + 2.0 ** -16 * size, "dx")
    within(g["dresidual"], d, (2.0 ** -8 if dtype is BF16 else 0) * abs(d) + 2.0 ** -16 * size, "dresidual")
    within(g["dw"], dw, 2.0 ** -15 * wsize, "dw")
    for _, flat, off in (dx, dr):
        assert untouched(flat, rows * D, off)


@pytest.mark.parametrize("rows,D", [(5, 9), (70, 37), (2500, 96), (7, 264), (2433, 1001), (3, 8200), (2, 16384)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_keep_to_themselves(rows, D, dtype):
    """A row of NaN changes no other row of any result."""
    def call(bad):
        x, r = slice_of((rows, D), 41, BF16, 1, 3), slice_of((rows, D), 42, dtype, 3, 1, 2.0)
        h, dout = at((rows, D), dtype, 1)[0], at((rows, D), BF16, 1)[0]
        h.copy_(rand((rows, D), 43, 2.0, F32))
        dout.copy_(rand((rows, D), 44))
        if bad is not None:
            x[bad] = dout[bad] = float("nan")
        w = 1 + rand((D,), 45, 0.2, F32)
        out, kept = pkg.add_rmsnorm(x, r, w)
        q, s, _ = pkg.add_rmsnorm_fp8(x, r, w)
        g = pkg.add_rmsnorm_backward(h, w, dout)
        return [out, kept, g["dx"], g["dresidual"], q.view(torch.uint8), s.view(torch.uint8)]

    want = call(None)
    for bad in {0, rows // 2, rows - 1}:
        got = call(bad)
        rest = torch.arange(rows, device=DEV) != bad
        assert all(torch.equal(a[rest], b[rest]) for a, b in zip(got, want))
        assert all(t[bad].isnan().all() for t in got[:4])
        assert (got[4][bad] & 0x7f == 0x7f).all() and (got[5][bad] == 255).all()


def test_in_place_at_odd_places():
    """h may be the stream itself and dx the stream's gradient, wherever they lie."""
    rows, D = 300, 1000
    for dtype in (BF16, F32):
        x, w = slice_of((rows, D), 51, BF16, 1, 3), 1 + rand((D,), 52, 0.2, F32)
        r = at((rows, D), dtype, 3)[0]
        r.copy_(rand((rows, D), 53, 2.0, F32))
        want, h = pkg.add_rmsnorm(x, r, w)
        out, same = pkg.add_rmsnorm(x, r, w, h=r)
        assert same is r and torch.equal(r, h) and torch.equal(out, want)
        dout, dh = rand((rows, D), 54), at((rows, D), dtype, 1)[0]
        dh.copy_(rand((rows, D), 55, 1.0, F32))
        a = pkg.add_rmsnorm_backward(r, w, dout, dh)
        b = pkg.add_rmsnorm_backward(r, w, dout, dh, grads=dict(dresidual=dh))
        assert b["dresidual"] is dh and all(torch.equal(a[n], b[n]) for n in a)
