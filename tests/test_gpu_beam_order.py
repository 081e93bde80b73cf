"""The order of la_beam_select's continuations where scores are equal: the lower (beam, token)
first.  Logits are equal as numbers (-0 and +0 are), so the expected orders are exact."""
import numpy as np
import pytest
import torch

import serving_ref as R
from gated_deltanet_recurrent_la_b200 import lastate as L
from test_gpu_beam_slots import select

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    L.lib()


def best(logits, cum, n_out, logits_dev=None):
    par, tok, _, _, _ = R.beam_ref(logits, cum.numpy(), None, -1, n_out)
    p, t, s, _ = select(logits, cum, None, -1, n_out, logits_dev)
    np.testing.assert_array_equal(p, par)
    np.testing.assert_array_equal(t, tok)
    return s


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,minus,plus,n_out", [(16, [0], [8], 1), (64, [0, 8], [32, 40], 2), (5000, [0], [2000], 1),
                                                (5001, [17], [16, 4999], 3), (33000, [5, 9000], [8, 8999, 32999], 4)])
def test_zeros_of_either_sign_tie(V, minus, plus, n_out, dtype):
    """The best of a piece is -0, that of a later one +0: the lower token comes first."""
    x = torch.full((1, 1, V), -1.0)
    x[..., minus] = -0.0
    x[..., plus] = 0.0
    best(x.to(dtype), torch.zeros(1, 1), n_out)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [61, 4999, 40001])
def test_zeros_of_either_sign_tie_by_whole_pieces(V, dtype):
    """Logits multiplied by a mask of 0 and 1: zeros of the logits' own signs, whole pieces of one."""
    gen = torch.Generator().manual_seed(V)
    sign = torch.randint(0, 2, (2, 3, (V + 7) // 8), generator=gen).repeat_interleave(8, -1)[..., :V] * 2.0 - 1.0
    keep = (torch.rand(2, 3, V, generator=gen) < 0.5) | (sign > 0)
    x = sign * torch.where(keep & (sign < 0), 1.0, 0.0)
    assert (x == 0).any() and x.max() == 0
    best(x.to(dtype), torch.tensor([[0.0, -0.25, -0.5]] * 2), 24)
