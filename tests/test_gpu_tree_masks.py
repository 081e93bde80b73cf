"""Drafted trees on q8 pools: masks that are wrong, and commits between two mask arrays."""
import numpy as np
import pytest
import torch

import serving_ref as R
from gated_deltanet_recurrent_la_b200 import lastate as L
from test_gpu_tree import commit, device, q8_pool, q8_values, run_tree

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    L.lib()


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (128, 128)])
def test_nothing_accepted_copies_the_tile_between_equal_masks(dk, dv):
    """Bit for bit, also where the two pools keep a mask array each."""
    inp = R.tree_inputs(lens=[3, 0, 5], Hqk=2, Hv=4, dk=dk, dv=dv, rule="gated_delta", state_dtype=F32, io_dtype=BF16, seed=23)
    src, _, mask = q8_pool(inp)
    u, leaf = torch.zeros(inp["T"], 4, dv), torch.tensor([-1, -1, -1], dtype=torch.int32)
    for m in (mask, mask.clone()):
        dst_t = torch.full((3,) + tuple(src.tensor.shape[1:]), 9, dtype=torch.uint8, device="cuda")
        assert commit(device(inp), src, L.Pool.q8(dst_t, 2, dk, dv, dk // 8, m), None, leaf, u) == 0
        assert torch.equal(dst_t, src.tensor[inp["read"].long().cuda()])


def flipped(mask, head):
    """The mask with one more row of `head`."""
    words = mask.cpu().numpy().view(np.uint32).copy()
    word = int(np.argmin(words[head] == 0xffffffff))
    low = next(i for i in range(32) if not words[head, word] >> i & 1)
    words[head, word] |= np.uint32(1 << low)
    return torch.tensor(words.view(np.int32)).cuda()


@pytest.mark.parametrize("rule", ["gated_delta", "kda"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_bad_q8_mask_skips_its_head(dk, dv, rule):
    inp = R.tree_inputs(lens=[9, 3], Hqk=2, Hv=4, dk=dk, dv=dv, rule=rule, state_dtype=F32, io_dtype=BF16, seed=12)
    good, _, mask = q8_pool(inp)
    clean_o, clean_u, err = run_tree(device(inp), good)
    assert err == 0
    bad = L.Pool.q8(good.tensor, inp["Hqk"], dk, dv, dk // 8, flipped(mask, 1))
    o, u, err = run_tree(device(inp), bad)
    assert err == L.DEVERR_Q8_MASK
    for h in range(4):
        if h == 1:
            assert torch.all(o[:, h] == 7.0) and torch.all(u[:, h] == 7.0)
        else:
            assert torch.equal(o[:, h], clean_o[:, h]) and torch.equal(u[:, h], clean_u[:, h])
    leaf, d = torch.tensor([8, -1], dtype=torch.int32), device(inp)
    dst_t = [torch.full((2,) + tuple(good.tensor.shape[1:]), 9, dtype=torch.uint8, device="cuda") for _ in range(3)]
    dst = [L.Pool.q8(t, inp["Hqk"], dk, dv, dk // 8, m) for t, m in zip(dst_t, (mask, mask, flipped(mask, 2)))]
    assert commit(d, good, dst[0], None, leaf, clean_u) == 0
    assert commit(d, bad, dst[1], None, leaf, clean_u) == L.DEVERR_Q8_MASK
    assert commit(d, good, dst[2], None, leaf, clean_u) == L.DEVERR_Q8_MASK
    for t, head in ((dst_t[1], 1), (dst_t[2], 2)):
        assert torch.all(t[:, head] == 9)
    others = [0, 2, 3]
    assert torch.equal(dst_t[1][:, others], dst_t[0][:, others])


@pytest.mark.parametrize("rule", ["linear", "gated_delta", "kda"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("io_dtype", [F32, BF16])
def test_commit_between_two_q8_masks(rule, dk, dv, io_dtype):
    """Rows change their kind and their place on the way, also where nothing is accepted."""
    inp = R.tree_inputs(lens=[3, 20, 1, 6, 2], Hqk=2, Hv=4, dk=dk, dv=dv, rule=rule, state_dtype=F32, io_dtype=io_dtype, seed=17)
    src, values, _ = q8_pool(inp, seed=1)
    other, _, mask = q8_pool({**inp, "pool": torch.zeros_like(inp["pool"])}, seed=2)
    u = torch.randn(inp["T"], 4, dv, generator=torch.Generator().manual_seed(3))
    leaf = torch.tensor([2, 13, -1, 5, -1], dtype=torch.int32)
    write = torch.tensor([6, 0, 3, 10, 8], dtype=torch.int32, device="cuda")
    before = other.tensor.clone()
    assert commit(device(inp), src, other, write, leaf, u) == 0
    ref, mag = R.commit_ref(inp, values, leaf, u)
    got = q8_values(other, write).double()
    # a code is off by half a step of its 32-column group (absmax / 127, itself within 2^-22), a BF16
    # row by 2^-8; FP32 sums of paths of at most 20 nodes before that
    group = ref.abs().reshape(5, 4, dk, dv // 32, 32).amax(-1, keepdim=True).expand(5, 4, dk, dv // 32, 32).reshape(ref.shape)
    words = mask.cpu().numpy().view(np.uint32)
    rows = torch.tensor([[bool(words[h, i // 32] >> (i % 32) & 1) for i in range(dk)] for h in range(4)])[None, :, :, None]
    step = torch.where(rows, 2.0 ** -8 * ref.abs(), group * (0.5 / 127 * (1 + 2.0 ** -10)))
    assert float(((got - ref).abs() - (step + 64 * 2.0 ** -24 * mag)).max()) <= 0
    rest = [s for s in range(other.tensor.shape[0]) if s not in write.tolist()]
    assert torch.equal(other.tensor[rest], before[rest])
