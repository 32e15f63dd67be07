"""Residual norm, rows in 8 bits and their scores against the float64 forms."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece
from encoder_reference import HALF, U, int8_rows, norm

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rows(n, d, dtype, seed=0, residual=True):
    g = torch.Generator().manual_seed(seed)
    t = [(torch.randn(n, d, generator=g) * (0.5 + 3 * torch.rand(n, 1, generator=g))).to(DT[dtype]) for _ in range(4)]
    return t[0], t[1] if residual else None, 1.0 + 0.3 * torch.randn(d, generator=g), t[2], t[3]


def near(got, want, tol):
    err = (got.double().cpu() - want).abs()
    assert torch.isfinite(got).all()
    worst = float((err / (tol + 1e-300)).max()) if err.numel() else 0.0
    print(f"  {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0


# every shape of a row: lanes 8, 16, 32, 64 (1, 2, 4 pieces), 256 (2, 4 pieces), and widths that fill none
WIDTHS = [8, 64, 72, 128, 256, 264, 512, 1000, 1024, 2048, 2056, 4096, 5000, 8192]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("residual", [True, False])
def test_norm_and_gradients(d, dtype, residual):
    n = 37
    print(f"[gpu] norm n={n} d={d} {dtype} residual={residual}", flush=True)
    x, r, w, dy, dh = rows(n, d, dtype, residual=residual)
    op = rece.ResidualNorm(n, d, eps=1e-5, dtype=dtype)
    X, W = x.cuda(), w.cuda()
    y, h, rstd = op.forward(X, None if r is None else r.cuda(), W)
    dx, dw = op.backward(dy.cuda(), h, W, rstd, dh=dh.cuda())
    want = norm(x, r, w, 1e-5, dy, dh)
    half = HALF[x.dtype]
    assert torch.equal(h.cpu(), want["h"])
    near(rstd, want["rstd"], 4 * U * want["rstd"])
    near(y, want["y"], (half + 6 * U) * want["y"].abs())
    H, g = want["h"].double(), dy.double() * w.double()
    rs = want["rstd"][:, None]
    # g h summed over a lane's pieces and a tree of lanes, then a handful of roundings
    c = (g * H).abs().mean(1, keepdim=True) * rs ** 2
    near(dx, want["dx"], half * want["dx"].abs() + U * (8 * rs * g.abs() + rs * H.abs() * c * (16 + 32) + 4 * dh.double().abs()))
    near(dw, want["dweight"], U * (n + 8) * (dy.double() * H * rs).abs().sum(0))
    y2, h2, rstd2 = op.forward(X, None if r is None else r.cuda(), W)
    dx2, dw2 = op.backward(dy.cuda(), h2, W, rstd2, dh=dh.cuda())
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_int8_rows(d, dtype):
    n = 41
    print(f"[gpu] int8 rows n={n} d={d} {dtype}", flush=True)
    x, r, w, _, _ = rows(n, d, dtype, seed=1)
    op = rece.ResidualNorm(n, d, eps=1e-6, dtype=dtype)
    y8, scale, h = op.forward_int8(x.cuda(), r.cuda(), w.cuda())
    want = norm(x, r, w, 1e-6)
    p = want["h"].double() * w.double()
    q, m = int8_rows(p)
    assert torch.equal(h.cpu(), want["h"]) and torch.equal(y8.cpu(), q)
    near(scale, m * want["rstd"], 4 * U * m * want["rstd"])
    x8, sx = rece.quantize_rows(x.cuda())
    q, m = int8_rows(x.double())
    assert torch.equal(x8.cpu(), q)
    near(sx, m, 2 * U * m)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("s,C,d", [(1, 1, 16), (1, 1000, 64), (5, 33, 128), (32, 4097, 48), (33, 129, 16), (128, 128, 128),
                                   (200, 1003, 64), (129, 257, 144), (300, 2000, 1040), (64, 300, 8192), (31, 31, 8192)])
def test_scores(s, C, d, dtype):
    print(f"[gpu] scores s={s} C={C} d={d} {dtype}", flush=True)
    g = torch.Generator().manual_seed(s + C + d)
    x8, y8 = (torch.randint(-128, 128, (n, d), generator=g, dtype=torch.int8) for n in (s, C))
    sx, sy = (torch.rand(n, generator=g) * 0.02 for n in (s, C))
    out = rece.Int8Scores(s, C, d, dtype=dtype).forward(x8.cuda(), sx.cuda(), y8.cuda(), sy.cuda())
    want = (x8.double() @ y8.double().T) * sx.double()[:, None] * sy.double()
    # the sum to float32, two products, the result
    near(out, want, (HALF[DT[dtype]] + 3 * U) * want.abs())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("s,C,d,shift", [
    (33, 1, 32, 0), (40, 63, 64, 1), (130, 64, 64, 0), (257, 65, 96, 3), (64, 127, 128, 2), (100, 1000, 256, 5),
    (129, 20001, 64, 7), (70, 30004, 112, 4), (2000, 997, 160, 1), (300, 4100, 272, 1),
])
def test_scores_at_any_address(s, C, d, shift, dtype):
    """Rows of results that begin anywhere in a line of memory; what lies around them stays."""
    print(f"[gpu] scores s={s} C={C} d={d} shift={shift} {dtype}", flush=True)
    g = torch.Generator().manual_seed(s + C + d)
    x8, y8 = (torch.randint(-128, 128, (n, d), generator=g, dtype=torch.int8) for n in (s, C))
    sx, sy = (torch.rand(n, generator=g) * 0.02 for n in (s, C))
    room = torch.full((s * C + shift + 256,), 7.0, dtype=DT[dtype], device="cuda")
    out = room[shift:shift + s * C].view(s, C)
    assert rece.Int8Scores(s, C, d, dtype=dtype).forward(x8.cuda(), sx.cuda(), y8.cuda(), sy.cuda(), out=out) is out
    want = (x8.double() @ y8.double().T) * sx.double()[:, None] * sy.double()
    near(out, want, (HALF[DT[dtype]] + 3 * U) * want.abs())
    assert (room[:shift] == 7.0).all() and (room[shift + s * C:] == 7.0).all()
