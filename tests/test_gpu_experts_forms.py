"""The experts' gradient with the row copy beside dx's product and clusters of
two CTA pairs in the same call (16384 rows or more, 256 an expert, K of 1024),
as a training batch takes them.  Formulas and tolerances of
test_gpu_experts_large."""
import pytest
import torch

from test_gpu_experts_large import _check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _dev(lib, cuda_ok):
    yield


@pytest.mark.parametrize("hidden,inner", [(512, 512), (1024, 520), (1280, 768)])
def test_copy_beside_clusters(hidden, inner):
    g = torch.Generator().manual_seed(hidden)
    idx = torch.rand(4200, 16, generator=g).argsort(1)[:, :4]
    _check(torch.where(torch.rand(4200, 4, generator=g) < 0.01, -1, idx), hidden, inner, 16)


def test_copy_beside_clusters_lopsided():
    g = torch.Generator().manual_seed(1)
    idx = torch.where(torch.rand(17000, 1, generator=g) < 0.9, 3, torch.randint(0, 9, (17000, 1), generator=g))
    _check(idx, 768, 640, 9, dtypes=(torch.bfloat16,))
