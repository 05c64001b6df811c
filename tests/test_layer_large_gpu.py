"""Tensors of more than 2^31 values: offsets that do not fit 32 bits, in the last rows of each."""
import pytest
import torch

import matrix_state_nonlinear_gb300 as pkg
from test_layer_gpu import BF16, DEV, F32, FP8, built, check_h  # noqa: F401

pytestmark = pytest.mark.gpu
OVER = 2 ** 31


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.get_device_properties(0).total_memory < 100 * 2 ** 30:
        pytest.skip("needs 100 GB")
    yield
    torch.cuda.empty_cache()


def fill(shape, seed, dtype=BF16):
    """Random rows, the same 4096 of them over and over (a bf16 randn of this size takes its time)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    some = torch.randn((4099, *shape[1:]), generator=g, device=DEV).to(dtype)
    t = torch.empty(shape, dtype=dtype, device=DEV)
    for i in range(0, shape[0], 4099):
        t[i:i + 4099] = some[:min(4099, shape[0] - i)]
    return t


def tail(t, n=5000):
    return t[-n:].contiguous()


def bits(t):
    return t.view(torch.uint8) if t.dtype.itemsize == 1 else t


def test_norm():
    rows, D = OVER // 2048 + 777, 2048
    x, r, w = fill((rows, D), 1), fill((rows, D), 2), torch.rand(D, device=DEV) + 0.5
    out, h = pkg.add_rmsnorm(x, r, w)
    a, b = pkg.add_rmsnorm(tail(x), tail(r), w)
    assert torch.equal(out[-5000:], a) and torch.equal(h[-5000:], b)
    # Few rows are spread over more threads, whose sums of squares are in another order.  Both results are within
    # 2^-8 + 2^-17 of the exact v (a rounding to bf16, float32 before it), so within 2^-7 + 2^-16 of v of each other,
    # and |v| is at most 1 + 2^-7 of either: (2^-7 + 2^-16)(1 + 2^-7) < 2^-7 + 2^-13.
    few = pkg.add_rmsnorm(x[:100], r[:100], w)[0].double()
    assert ((out[:100].double() - few).abs() <= (2.0 ** -7 + 2.0 ** -13) * few.abs()).all()
    q, s, h = pkg.add_rmsnorm_fp8(x, r, w, h=h)
    a, c, _ = pkg.add_rmsnorm_fp8(tail(x), tail(r), w)
    assert torch.equal(bits(q[-5000:]), bits(a)) and torch.equal(bits(s[-5000:]), bits(c))
    del q, s, out
    g = pkg.add_rmsnorm_backward(h, w, x, r)
    b = pkg.add_rmsnorm_backward(tail(h), w, tail(x), tail(r))
    assert torch.equal(g["dx"][-5000:], b["dx"])
    inv = torch.rsqrt(h[:4099].float().square().mean(1, keepdim=True) + 1e-5)
    period = (x[:4099].double() * h[:4099].double() * inv.double())  # rows repeat: whole periods and a rest
    whole, rest = divmod(rows, 4099)
    want = period.sum(0) * whole + period[:rest].sum(0)
    # every term within 2^-17 (inv), summed by 608 blocks of some 1700 rows: 2^-13 of the magnitudes' sum
    size = period.abs().sum(0) * whole + period[:rest].abs().sum(0)
    assert ((g["dw"].double() - want).abs() <= 2.0 ** -13 * size).all()


def test_norm_of_odd_rows():
    """Rows that start anywhere; a multiple of 8 of them before the last 5000, which so start as they do alone."""
    rows, D = (OVER // 2049 + 777) // 8 * 8, 2049
    x, r, w = fill((rows, D), 6), fill((rows, D), 7), torch.rand(D, device=DEV) + 0.5
    out, h = pkg.add_rmsnorm(x, r, w)
    a, b = pkg.add_rmsnorm(tail(x), tail(r), w)
    assert torch.equal(out[-5000:], a) and torch.equal(h[-5000:], b)
    del out
    q, s, h = pkg.add_rmsnorm_fp8(x, r, w, h=h)
    a, c, _ = pkg.add_rmsnorm_fp8(tail(x), tail(r), w)
    assert torch.equal(bits(q[-5000:]), bits(a)) and torch.equal(bits(s[-5000:]), bits(c))
    del q, s
    g = pkg.add_rmsnorm_backward(h, w, x, r)
    assert torch.equal(g["dx"][-5000:], pkg.add_rmsnorm_backward(tail(h), w, tail(x), tail(r))["dx"])


@pytest.mark.parametrize("D", [2048, 2047])
def test_quantise(D):
    rows = OVER // D + 99
    x = fill((rows, D), 3)
    q, s = pkg.quantise_fp8(x)
    a, b = pkg.quantise_fp8(tail(x))
    assert torch.equal(bits(q[-5000:]), bits(a)) and torch.equal(bits(s[-5000:]), bits(b))


def test_linear():
    M, N, K = OVER // 8200 + 300, 8200, 136
    x = fill((M, K), 4)
    w = pkg.quantise_weight_fp8(fill((N, K), 5))
    out = pkg.linear_fp8(x, None, *w)
    want = pkg.linear_fp8(tail(x), None, *w)
    assert torch.equal(out[-5000:], want) and torch.equal(out[:300], pkg.linear_fp8(x[:300], None, *w))
    assert pkg.stream_status() == 0


def test_clip():
    n = OVER + 12345
    g = [torch.ones(1000, dtype=F32, device=DEV), torch.full((n,), 0.5, dtype=BF16, device=DEV)]
    norm = pkg.clip_grad_norm(g, 1.0)
    want = (1000 + 0.25 * n) ** 0.5
    assert abs(float(norm) - want) < 2.0 ** -21 * want
    by = torch.tensor(0.5 / want).to(BF16)  # within 2^-22 of the factor: the same bf16 but next to a border
    for part in (g[1][:100000], g[1][-100000:]):
        assert ((part.float() - 0.5 / want).abs() <= (2.0 ** -8 + 2.0 ** -20) * 0.5 / want).all() and (part == part[0]).all()
    assert g[1][0] == g[1][-1] and abs(float(g[1][0]) - float(by)) <= 2.0 ** -7 * float(by)
