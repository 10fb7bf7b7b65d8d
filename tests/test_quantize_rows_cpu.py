"""quantize_rows: e4m3 rows with scales, down to fp32's smallest values."""
import pytest
import torch

from multiresolution_hash_grid_amd import quantize_rows

TINY = 2.0 ** -149


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_are_within_a_code_of_their_values(dtype):
    g = torch.Generator().manual_seed(0)
    powers = torch.tensor([2.0, 0.0, -20.0, -35.0, -36.0, -38.0, -40.0, -42.0, -44.0, -45.0], dtype=torch.float64)
    w = (torch.randn(10, 77, generator=g, dtype=torch.float64) * 10 ** powers[:, None])
    w[:, ::5] = 0
    w = torch.cat([w, torch.zeros(1, 77, dtype=torch.float64)]).to(dtype)
    q, scale = quantize_rows(w)
    got, sc, want = q.float().double(), scale.double(), w.double()
    assert got.isfinite().all() and sc.isfinite().all() and not got[want == 0].any() and not got[sc == 0].any()
    assert ((sc - want.abs().amax(1) / 448).abs() <= 2.0 ** -23 * sc + TINY).all()
    # half a code's step, the roundings of scale and quotient, and the scale's own step (448 times at most) where it is tiny
    err = want.abs() * (2.0 ** -4 + 2.0 ** -21) + 2.0 ** -10 * sc[:, None] + 448 / 2 * TINY
    assert ((got * sc[:, None] - want).abs() <= err).all()


def test_ordinary_rows_round_as_before():
    w = torch.randn(300, 64, generator=torch.Generator().manual_seed(1))
    q, scale = quantize_rows(w)
    want = w.abs().amax(1) / 448.0
    assert torch.equal(scale, want)
    assert torch.equal(q.view(torch.uint8), (w * (1.0 / want)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
