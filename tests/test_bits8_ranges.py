"""The 8-bit decode operators where values lie at the ends of their types or far apart, against the definitions in 64 bits
(bits8_util)."""
import math

import pytest
import torch

import bits8_util as U
import layer_embedding_lookup_amd as ple
import test_bits8_gpu as G
import test_bits8_kernels as K

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F64, BF, I32 = torch.float64, torch.bfloat16, torch.int32


# ---- norm ----

# powers of two that inputs and weights are of: products from fp32's normal numbers down past its least one
TINY = [(-50, -40), (-50, -52), (-64, -62), (-64, -64), (-66, -64), (-70, -62), (-120, -12), (-20, -112), (-100, -60), (-120, -100),
        (-126, -126), (-131, 0), (0, -131), (-131, 100), (60, -131)]


def check_tiny(x, w, res, eps, got):
    """As G.check_norm, but for the scales, which fp32 rounds by up to half of its least step, 2^-150, where they are below
    its normal numbers."""
    codes, scales, h = got
    want, want_scales, want_h = U.norm8(x, w, res, eps)
    assert torch.equal(codes.cpu().to(F64), want)
    bad = torch.isnan(want_scales)                            # (rows whose squares leave fp32's range)
    assert torch.equal(torch.isnan(scales.cpu()), bad)
    assert ((scales.cpu().to(F64) - want_scales).abs() <= 60 * 2.0 ** -24 * want_scales + 2.0 ** -149)[~bad].all()
    if res is not None:
        assert torch.equal(h.cpu().to(F64), want_h)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("N", [16, 512, 2064, 4096, 8208, 20000])
def test_norm_rows_whose_products_underflow(N, residual):
    """Every row has the codes of its exact quotients, however small its products, beside rows of ordinary size."""
    for a, b in TINY:
        g = G.gen(N + a - b)
        x = torch.randn((6, N), generator=g).double() * 2.0 ** a
        x[1] = torch.randn(N, generator=g)                    # an ordinary row, if the weight is not tiny
        x[4] = 0
        x[5] *= torch.pow(2.0, torch.randint(-4, 5, (N,), generator=g).double())
        x = x.to(BF)
        w = (torch.randn(N, generator=g).double() * 2.0 ** b).to(BF)
        res = (torch.randn((6, N), generator=g).double() * 2.0 ** (a - 1)).to(BF) if residual else None
        if residual:
            res[4] = 0
        got = ple.ple_rms_norm8(x.to(DEV), w.to(DEV), residual=None if res is None else res.to(DEV))
        check_tiny(x, w, res, 1e-6, got)
        assert (got[0][4] == 0).all() and got[1][4] == 0
        assert got[0].abs().amax(1).tolist() == [0 if s != s or s == 0 else 127 for s in U.norm8(x, w, res, 1e-6)[1].tolist()]


def test_norm_tiny_rows_in_place_and_strided():
    for N in (48, 4096, 20000):
        g = G.gen(N)
        wide = torch.full((5, N + 16), math.nan).to(BF)
        wide[:, 8:N + 8] = (torch.randn((5, N), generator=g).double() * 2.0 ** -70).to(BF)
        x, w = wide[:, 8:N + 8], (torch.randn(N, generator=g).double() * 2.0 ** -62).to(BF)
        check_tiny(x, w, None, 1e-6, ple.ple_rms_norm8(wide.to(DEV)[:, 8:N + 8], w.to(DEV)))
        x = x.contiguous()
        res = (torch.randn((5, N), generator=g).double() * 2.0 ** -70).to(BF)
        for into in ("x", "residual"):
            dx, dres = x.to(DEV), res.to(DEV)
            got = ple.ple_rms_norm8(dx, w.to(DEV), residual=dres, residual_out=dx if into == "x" else dres)
            check_tiny(x, w, res, 1e-6, got)


@pytest.mark.parametrize("N", [16, 512, 2064, 4096, 8208, 20000])
def test_norm_weights_of_no_number(N):
    """A NaN or an infinity in the weight is in every row's products, as 0 * infinity too: scales of NaN, codes of zero, the
    residual as ever."""
    g = G.gen(N)
    x, res = torch.randn((5, N), generator=g).to(BF), torch.randn((5, N), generator=g).to(BF)
    x[3] = res[3] = 0
    for at in (0, 7, N // 2, N - 1):
        x[1, at] = res[1, at] = 0
        for value in (math.nan, -math.nan, math.inf, -math.inf):
            w = torch.randn(N, generator=g).to(BF)
            w[at] = value
            for r in (None, res):
                codes, scales, h = ple.ple_rms_norm8(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV))
                assert torch.isnan(scales).all() and (codes == 0).all()
                assert r is None or torch.equal(h.cpu(), (x.float() + r.float()).to(BF))


@pytest.mark.parametrize("N", [48, 4096, 20000])
def test_norm_scales_whose_products_overflow(N):
    """A largest product below fp32's 127th part, times a norm's factor far above 127: the scale itself is in range."""
    g = G.gen(N)
    x = (torch.randn((4, N), generator=g).clamp(-4, 4).double() * 2.0 ** -9).to(BF)
    x[:, 3] = 2.0 ** -7
    w = (torch.rand(N, generator=g).double() * 2.0 ** 126).to(BF)
    w[3] = 2.0 ** 127
    top = (x.double() * w.double()).abs().amax(1)
    factor = 1 / (x.double().square().mean(1) + 1e-6).sqrt()
    assert (127 * top < 3.4e38).all() and (top * factor > 3.5e38).all()
    got = ple.ple_rms_norm8(x.to(DEV), w.to(DEV))
    G.check_norm(x, w, None, 1e-6, got)
    assert torch.isfinite(got[1]).all()
