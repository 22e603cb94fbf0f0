"""GPU parity of the RMS norm on rows whose squares lie outside fp32's range.  The plain implementation and the
tolerance of a bf16 result are those of test_step_gpu.py."""

import pytest
import torch

from tests import step_reference as ref
from tests.test_step_gpu import BF, DEV, F32, bd, check_bf16, check_e4m3, on_gpu, same_bits  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [8, 512, 520, 4096, 6152, 8200, 16384, 20000, 32768, 65536])
@pytest.mark.parametrize("x_t,res_t", [(F32, None), (BF, None), (F32, BF), (BF, F32)])
def test_squares_past_fp32(bd, d, x_t, res_t):
    """Rows of values from 2^-149 to 2^127, alone and mixed, with and without an eps that covers small ones: the mean of
    their squares has a root in fp32 though the squares have no place there.  Rows of ordinary size between them are
    bitwise what they are alone."""
    print("norm range", d, x_t, res_t, flush=True)
    gen = torch.Generator().manual_seed(d)
    sizes = [2.0 ** 120, 1.0, 2.0 ** 70, 2.0 ** 64, 2.0 ** 50, 2.0 ** -30, 2.0 ** -62, 2.0 ** -75, 2.0 ** -100,
             2.0 ** -120, 2.0 ** 49, 2.0 ** -33]
    x = torch.randn((len(sizes), d), generator=gen) * torch.tensor(sizes)[:, None]
    x[2, 1::2] = 0.5                      # what is small in a row of large values stays so
    x[3, : d // 2] *= 2.0 ** -60
    x[6, 0] = 2.0 ** -20                  # one larger value in a small row
    x = x.to(x_t)
    res = torch.randn((len(sizes), d), generator=gen) * torch.tensor(sizes)[:, None]
    res = None if res_t is None else res.to(res_t)
    gain = (1 + 0.3 * torch.randn((2, d), generator=gen)).to(BF if d % 16 else F32)
    ids = torch.arange(len(sizes), dtype=torch.int32) % 2
    gx, gr, gg, gi = on_gpu(x, res, gain, ids)
    for eps in (1e-5, 0.0, 1e-20, 1e-30):
        want, res_want = ref.rms_norm(x, gain, float(torch.tensor(eps)), res, ids)
        got = bd.bd_rms_norm(gx, gg, eps, residual=gr, variant_ids=gi)
        y = got if res is None else got[0]
        check_bf16(y, want, d)
        if res is not None:
            assert same_bits(got[1], res_want)
            inplace = gr.clone()
            again = bd.bd_rms_norm(gx, gg, eps, residual=inplace, variant_ids=gi, residual_out=inplace)
            assert same_bits(again[0], y) and same_bits(inplace, res_want)
        one = bd.bd_rms_norm(gx[1:2], gg, eps, residual=None if gr is None else gr[1:2], variant_ids=gi[1:2])
        assert same_bits(y[1:2], one if res is None else one[0])
        codes, scales, *_ = bd.bd_rms_norm_e4m3(gx, gg, eps, residual=gr, variant_ids=gi)
        check_e4m3(codes, scales, want, d)


@pytest.mark.parametrize("d", [64, 4096, 8200])
def test_specials_among_large_values(bd, d):
    """An id out of range, NaN and infinities in rows of large values, and rows of zeros with eps 0."""
    x = torch.full((6, d), 2.0 ** 100)
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    x[4] = 0
    x[5] = -2.0 ** -140
    gain = torch.ones((1, d))
    ids = torch.tensor([0, 0, 0, 1, 0, 0], dtype=torch.int32)
    y = ref.to64(bd.bd_rms_norm(x.to(DEV), gain.to(DEV), 0.0, variant_ids=ids.to(DEV)))
    assert (abs(y[0] - 1) <= 2.0 ** -8).all() and (abs(y[5] + 1) <= 2.0 ** -8).all()
    nan = y != y
    assert nan[1].all() and nan[3].all() and nan[4].all()
    assert nan[2, 5] and (y[2][~nan[2]] == 0).all() and nan[2].sum() == 1


@pytest.mark.parametrize("d", [8, 520, 8192, 65536])
def test_squares_next_to_the_borders(bd, d):
    """Rows of one size on either side of where a row is scaled, at the ends of fp32's range, and with eps near them."""
    sizes = [s * 2.0 ** e for e in (-149, -148, -126, -90, -41, -40, -39, -31, -30, -29, 49, 50, 51, 56, 63, 64, 127)
             for s in (1.0, 1.5, 1.75) if s * 2.0 ** e >= 2.0 ** -148 or s == 1.0]
    x = torch.tensor(sizes, dtype=torch.float64).float()[:, None].repeat(1, d)
    x[:, 1::2] *= -1
    gain = torch.full((1, d), 1.25)
    for eps in (0.0, 2.0 ** -80, 2.0 ** -81, 2.0 ** 100, 2.0 ** 101, 2.0 ** -149):
        want, _ = ref.rms_norm(x, gain, eps)
        check_bf16(bd.bd_rms_norm(x.to(DEV), gain.to(DEV), eps), want, d)
