"""The residual norm on more rows than its grids take at once (2,048 workgroups forward, 1,024 back, of 1 to 32 rows): every
row's results and the sums over all of them."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece
from encoder_reference import HALF, U, int8_rows, norm
from test_gpu_norm_scores import DT, near, rows

pytestmark = pytest.mark.gpu


def dweight_error(dw, dy, h, rstd):
    """Norm of dweight's error in units of U times the root of its terms' squares."""
    terms = dy.double() * h.double() * rstd[:, None]
    return float((dw.double() - terms.sum(0)).norm() / (U * terms.square().sum().sqrt()))


# A term takes roundings of rstd (three: its argument, root and quotient) and of h rstd, the sums one of a workgroup's part
# and one of the result: six of at most U, uniform, independent over the terms: U sqrt(6 / 3) = 1.4 U.
MOST = 2.0


# 3 rounds forward (65,536, 16,384 and 2,048 rows each), the last one in part; 5, 3 and 5 back
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(150037, 64), (20001, 256), (5003, 4096)])
def test_rows_in_many_rounds(n, d, dtype):
    print(f"[gpu] norm rounds n={n} d={d} {dtype}", flush=True)
    x, r, w, dy, dh = rows(n, d, dtype)
    op = rece.ResidualNorm(n, d, eps=1e-5, dtype=dtype)
    X, R, W = x.cuda(), r.cuda(), w.cuda()
    y, h, rstd = op.forward(X, R, W)
    dx, dw = op.backward(dy.cuda(), h, W, rstd, dh=dh.cuda())
    want = norm(x, r, w, 1e-5, dy, dh)
    half = HALF[x.dtype]
    assert torch.equal(h.cpu(), want["h"])
    near(rstd, want["rstd"], 4 * U * want["rstd"])
    near(y, want["y"], (half + 6 * U) * want["y"].abs())
    H, g, rs = want["h"].double(), dy.double() * w.double(), want["rstd"][:, None]
    c = (g * H).abs().mean(1, keepdim=True) * rs ** 2
    near(dx, want["dx"], half * want["dx"].abs() + U * (8 * rs * g.abs() + rs * H.abs() * c * (16 + 32) + 4 * dh.double().abs()))
    off = dweight_error(dw.cpu(), dy, want["h"], want["rstd"])
    print(f"  dweight: {off:.2f} U")
    assert off <= MOST
    y8, scale, h8 = op.forward_int8(X, R, W)
    q, m = int8_rows(H * w.double())
    assert torch.equal(h8, h) and torch.equal(y8.cpu(), q)
    near(scale, m * want["rstd"], 4 * U * m * want["rstd"])
    x8, sx = rece.quantize_rows(X)
    q, m = int8_rows(x.double())
    assert torch.equal(x8.cpu(), q)
    near(sx, m, 2 * U * m)


@pytest.mark.parametrize("n,d", [(2_000_003, 64), (250_007, 512), (20_011, 8192)])
def test_weight_gradient_of_many_rows(n, d):
    print(f"[gpu] dweight n={n} d={d}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    h, dy = (torch.randn(n, d, generator=g, device="cuda") for _ in range(2))
    w = torch.rand(d, generator=g, device="cuda")
    op = rece.ResidualNorm(n, d, dtype="f32")
    _, _, rstd = op.forward(h, None, w)
    _, dw = op.backward(dy, h, w, rstd)
    exact = 1.0 / (h.double().square().mean(1) + 1e-6).sqrt()
    off = dweight_error(dw, dy, h, exact)
    print(f"  dweight: {off:.2f} U")
    assert off <= MOST


def test_weight_gradient_beyond_two_to_the_31_elements():
    n, d = 290_003, 8192
    g = torch.Generator(device="cuda").manual_seed(0)
    h, dy = (torch.randn(n, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = torch.rand(d, generator=g, device="cuda")
    op = rece.ResidualNorm(n, d)
    print(f"[gpu] dweight n={n} d={d}", flush=True)
    _, _, rstd = op.forward(h, None, w)
    _, dw = op.backward(dy, h, w, rstd)
    total, squares = torch.zeros(d, dtype=torch.float64, device="cuda"), 0.0
    for a in range(0, n, 20_000):
        x = h[a:a + 20_000].double()
        terms = dy[a:a + 20_000].double() * x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt()
        total += terms.sum(0)
        squares += float(terms.square().sum())
    off = float((dw.double() - total).norm()) / (U * squares ** 0.5)
    print(f"  dweight: {off:.2f} U")
    assert off <= MOST
