"""The norm's output in 8 bits where y / scale lies between two e4m3 numbers: bit by bit the quotient's own rounding."""
import numpy as np
import pytest
import torch

import long_fft_convolution_amd as fc

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _weights(m, dtype):
    """Weights of largest 7 m / 1024, whose scale is m 2^-16: every halfway point of two e4m3 numbers that the type holds
    times that scale, and neighbours of them."""
    ties = np.concatenate([(np.arange(8, 16) + 0.5) * 2.0 ** e for e in range(-8, 6)] + [(np.arange(8) + 0.5) * 2.0 ** -9])
    w = torch.from_numpy(np.concatenate([ties[ties < 448] * m * 2.0 ** -16, [7 * m / 1024], ties[:40] * m * 2.0 ** -15]))
    w = w[w <= 7 * m / 1024]
    w = torch.cat([w[w == w.to(DT[dtype]).double()], w * (1 + 2.0 ** -6)]).clamp(max=7 * m / 1024).to(DT[dtype])
    return torch.cat([w, w[:1].expand(-len(w) % 16)])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m", [7, 13, 14, 15, 21, 27])
@pytest.mark.parametrize("copies,odd", [(1, 0), (1, 1), (40, 0), (9, 3)])
def test_quotients_between_two_numbers(m, copies, odd, dtype):
    """Rows of +-1 with eps = 0: their root mean square is 1 and y the weight itself, exactly."""
    w = _weights(m, dtype).repeat(copies)
    w = w[:len(w) - odd]
    signs = torch.randint(0, 2, (5, len(w)), generator=torch.Generator().manual_seed(m)) * 2 - 1
    out, scales = fc.rms_norm(signs.to(DT[dtype]).cuda(), w.cuda(), eps=0.0, eight_bits=True)
    y = (signs.float() * w.float()).numpy()
    scale = np.float32(np.abs(y).max()) / np.float32(448)
    assert (scales.cpu().numpy() == scale).all()
    want = torch.from_numpy(np.divide(y, scale)).to(torch.float8_e4m3fn)
    same = out.cpu().view(torch.uint8) == want.view(torch.uint8)
    assert same.all(), f"{(~same).sum()} of {same.numel()}, the first {y.ravel()[int((~same).ravel().nonzero()[0])]!r} / {scale!r}"


def test_rows_with_an_infinity():
    """The scale is infinite: finite values are 0 and infinite ones NaN, as y / scale is."""
    x = torch.randn((3, 256), generator=torch.Generator().manual_seed(1))
    w = torch.ones(256)
    w[7] = float("inf")
    out, scales = fc.rms_norm(x.cuda(), w.cuda(), eight_bits=True)
    out = out.float().cpu()
    assert torch.isinf(scales).all() and torch.isnan(out[:, 7]).all() and (out[:, :7] == 0).all() and (out[:, 8:] == 0).all()
