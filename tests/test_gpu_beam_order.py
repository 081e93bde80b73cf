"""The order of la_beam_select's continuations where scores are equal, and its use in place.

Equal scores go to the lower (beam, token).  Two logits are equal as numbers (-0 and +0 are), and
two beams with the same logits and the same cum_score have the same scores wherever their rows
lie in memory, so the expected orders are exact."""
import numpy as np
import pytest
import torch

import serving_ref as R
from gated_deltanet_recurrent_la_b200 import lastate as L
from test_gpu_beam_slots import beam_inputs, i32, select

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


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,K,V", [(3, 4, 5), (2, 8, 97), (2, 4, 4099), (1, 5, 9001), (1, 2, 50257), (40, 8, 5003)])
def test_equal_beams_tie(B, K, V, dtype):
    """Rows with the same logits start at every alignment when the vocabulary is odd."""
    x, _ = beam_inputs(B, 1, V, dtype, seed=V)
    best(x.expand(B, K, V).contiguous(), torch.full((B, K), -1.375), min(2 * K, V))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_equal_pairs_of_beams_tie(dtype):
    """Beams 0 and 3, and 1 and 2, have the same logits and cum_score."""
    x, _ = beam_inputs(4, 2, 10007, dtype, seed=2)
    best(x[:, [0, 1, 1, 0]].contiguous(), torch.tensor([[-0.5, -0.75, -0.75, -0.5]] * 4), 12)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [1000, 30011])
def test_scores_do_not_depend_on_where_a_row_lies(V, dtype):
    """The same rows at every offset: the same bits."""
    B, K = 1, 3
    x, cum = beam_inputs(B, K, V, dtype, seed=V + 1)
    scores = []
    for offset in range(9):
        flat = torch.full((offset + B * K * (V + 3) + 16,), 1e9, dtype=dtype, device="cuda")
        view = flat[offset:offset + B * K * (V + 3)].view(B, K, V + 3)[:, :, :V]
        view.copy_(x)
        scores.append(best(x, cum, 7, logits_dev=view))
    assert all(np.array_equal(s, scores[0]) for s in scores)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("seed", range(3))
def test_in_place(seed, dtype):
    """score over cum_score and finished_out over finished, with as many continuations as beams."""
    B, K, V, eos = 12, 8, 301, 7
    x, cum = beam_inputs(B, K, V, dtype, seed=seed, masked=0.0)
    fin = (torch.rand(B, K, generator=torch.Generator().manual_seed(seed)) < 0.4).to(torch.int32)
    par, tok, sc, fo, gap = R.beam_ref(x, cum.numpy(), fin.numpy(), eos, K)
    assert gap > 1e-5
    parent, token, c, f = i32(np.zeros((B, K))), i32(np.zeros((B, K))), cum.cuda(), fin.cuda()
    ws = torch.empty(L.la_beam_workspace_bytes(B, K, V, K), dtype=torch.uint8, device="cuda")
    L.check(L.la_beam_select(x.cuda(), c, f, eos, parent, token, c, f, ws))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(parent.cpu().numpy(), par)
    np.testing.assert_array_equal(token.cpu().numpy(), tok)
    np.testing.assert_array_equal(f.cpu().numpy(), fo)
    s = c.cpu().numpy()
    assert np.all(np.abs(s - sc) <= 2.0 ** -20 + 2.0 ** -23 * np.abs(sc))
