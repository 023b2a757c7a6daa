"""GPU: the int8 product of few rows with very many channels, bit for bit against sums in 64-bit integers."""
import pytest
import torch

from test_gpu_int8_gemm import TYPES, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [16, 32, 33, 64, 65, 100, 128, 129])
@pytest.mark.parametrize("O,H", [(32832, 80), (65543, 272), (131072, 64)])
def test_one_band_of_rows(T, O, H):
    """Row tiles follow the rows there are, however many channels: tiles of 64 up to 64 rows, of 128 up to 128."""
    check(T, O, H, torch.bfloat16, T + H)


@pytest.mark.parametrize("dt", TYPES)
def test_one_band_of_rows_in_all_types(dt):
    for T in (48, 100):
        check(T, 70001, 144, dt, 3)
