"""Long paths of drafted trees whose far nodes weigh as much as the near ones (no gates, or gates
close to 1 in magnitude), in every operand form.

Bounds.  BF16 q, k, v are multiplied exactly and FP32 factors to 2^-23 of a product; the rest is
FP32 in sums of as many terms as those of the elementary recurrence, so that the error against 64
bits, over all outputs, is held to three times that of elementary FP32.  A BF16 output adds half a
step, 2^-8 of its value."""
import pytest
import torch

import serving_ref as R
from gated_deltanet_recurrent_la_b200 import lastate as L
from test_gpu_serving_edges import recurrence_fp32
from test_gpu_tree import device, q8_pool, run_tree

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    L.lib()


def long_inputs(rule, n, shape, dk, dv, state_dtype, io_dtype, seed):
    inp = R.tree_inputs(lens=[n, n - 2], Hqk=1, Hv=2, dk=dk, dv=dv, rule=rule, state_dtype=state_dtype, io_dtype=io_dtype,
                        seed=seed, shape=shape)
    gen = torch.Generator().manual_seed(seed + 1)
    g = inp["g"]
    inp["g"] = (1 - torch.rand(g.shape, generator=gen) * 2.0 ** -6) * (torch.randint(0, 2, g.shape, generator=gen) * 2 - 1)
    return inp


def as_near_as_fp32(inp, states, pool=None):
    """states: what the pool holds, [slots, Hv, dk, dv]."""
    at = {**inp, "pool": states}
    o_ref, u_ref, _, _, _ = R.tree_ref(at, states)
    o32, u32 = recurrence_fp32(at)
    o, u, err = run_tree(device(inp), pool)
    assert err == 0
    mine, theirs = (float((x.double() - u_ref).norm() / u_ref.norm()) for x in (u, u32))
    assert mine <= 3 * theirs + 2.0 ** -30, (mine, theirs)
    theirs = float((o32.double() - o_ref).norm())
    if o.dtype == F32:
        mine = float((o.double() - o_ref).norm())
        assert mine <= 3 * theirs + 2.0 ** -30 * float(o_ref.norm()), (mine, theirs)
    else:  # no element's FP32 error is above the norm of all of them
        fp32 = 3 * theirs + 2.0 ** -30 * float(o_ref.norm())
        assert float(((o.double() - o_ref).abs() - (2.0 ** -8 * (o_ref.abs() + fp32) + fp32)).max()) <= 0


@pytest.mark.parametrize("n", [33, 48, 57, 64])
@pytest.mark.parametrize("shape", ["chain", "tree"])
@pytest.mark.parametrize("rule", ["linear", "delta", "gated", "gated_delta", "kda"])
@pytest.mark.parametrize("state_dtype,io_dtype", [(BF16, BF16), (F32, BF16), (BF16, F32)])
def test_far_nodes_of_a_path(state_dtype, io_dtype, rule, shape, n):
    inp = long_inputs(rule, n, shape, 128, 128, state_dtype, io_dtype, seed=n)
    as_near_as_fp32(inp, inp["pool"])


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64)])
@pytest.mark.parametrize("rule", ["linear", "delta", "kda"])
def test_far_nodes_of_a_path_narrow_heads(rule, dk, dv):
    inp = long_inputs(rule, 64, "chain", dk, dv, BF16, BF16, seed=dk + dv)
    as_near_as_fp32(inp, inp["pool"])


@pytest.mark.parametrize("n", [40, 64])
@pytest.mark.parametrize("rule", ["linear", "delta", "gated_delta", "kda"])
@pytest.mark.parametrize("io_dtype", [F32, BF16])
def test_far_nodes_of_a_path_q8_state(io_dtype, rule, n):
    inp = long_inputs(rule, n, "chain", 128, 128, F32, io_dtype, seed=n + 5)
    pool, values, _ = q8_pool(inp)
    as_near_as_fp32(inp, values, pool)
