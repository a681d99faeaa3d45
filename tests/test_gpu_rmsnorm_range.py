"""RMS norm's 8-bit output of very large values: every step scales by the powers
of two exactly, so the codes must be those of the same values times 2^-100."""
import pytest
import torch

from newton_schulz_gb300 import binding as B

pytestmark = pytest.mark.gpu
F32, E4M3 = torch.float32, torch.float8_e4m3fn
EPS = 1e-6


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield


def _rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("group", [0, 128])
def test_e4m3_of_very_large_values(group):
    # values up to 2^127 and their scales are normal f32 numbers: codes as for small ones
    x = _rand((9, 256), F32, 5)
    gain = torch.full((256,), 1.2e37, device="cuda")
    y, _, s = B.muon_rmsnorm_forward(x, gain, eps=EPS, y_dtype=E4M3, group=group)
    small, _, t = B.muon_rmsnorm_forward(x, gain * 2.0 ** -100, eps=EPS, y_dtype=E4M3, group=group)
    assert torch.equal(y.float(), small.float()) and torch.equal(s, t * 2.0 ** 100)
    big = torch.full((256,), 8e37, device="cuda")
    y, _, s = B.muon_rmsnorm_forward(x.clamp(-2, 2), big, eps=EPS, y_dtype=E4M3, group=group)
    small, _, t = B.muon_rmsnorm_forward(x.clamp(-2, 2), big * 2.0 ** -100, eps=EPS, y_dtype=E4M3, group=group)
    assert float(s.max()) * 448 > 2.0 ** 126 and torch.equal(y.float(), small.float())
    assert torch.equal(s, t * 2.0 ** 100)
