"""Arrays of the serving operators that end before the nodes do: the offsets are checked against
the shortest one on the device, so that nothing behind it is read."""
import numpy as np
import pytest
import torch

import serving_ref as R
from gated_deltanet_recurrent_la_b200 import lastate as L
from test_gpu_tree import commit, device, run_tree

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    L.lib()


@pytest.mark.parametrize("longer", [0, 5])
def test_parents_that_end_before_the_rows(longer):
    """Rows behind the last node (a padded batch) are left alone; a sequence whose nodes have no
    parents in the array is skipped."""
    inp = R.tree_inputs(lens=[5, 6, 7], Hqk=1, Hv=2, dk=128, dv=128, rule="gated_delta", state_dtype=BF16, io_dtype=BF16, seed=1)
    clean_o, clean_u, err = run_tree(device(inp))
    assert err == 0
    pad = lambda x: torch.cat([x, torch.full((longer, *x.shape[1:]), float("nan"), dtype=x.dtype)])  # noqa: E731
    wide = {**inp, **{x: pad(inp[x]) for x in ("q", "k", "v", "g", "beta")}, "T": inp["T"] + longer}
    o, u, err = run_tree(device(wide))
    assert err == 0 and torch.equal(o[:18], clean_o) and torch.equal(u[:18], clean_u) and torch.all(o[18:] == 7.0)
    short = {**wide, "parent": inp["parent"][:17].clone()}
    o, u, err = run_tree(device(short))
    assert err == L.DEVERR_CU_SEQLENS and torch.equal(o[:11], clean_o[:11]) and torch.all(o[11:] == 7.0)
    d, dst = device(short), torch.full((3, 2, 128, 128), 3.0, dtype=BF16, device="cuda")
    leaf = torch.tensor([4, 5, 6], dtype=torch.int32)
    assert commit(d, L.Pool(d["pool"], 1), L.Pool(dst, 1), None, leaf, clean_u) == L.DEVERR_CU_SEQLENS
    assert torch.all(dst[2] == 3.0) and not torch.any(torch.all(dst[:2].flatten(1) == 3.0, dim=1))


@pytest.mark.parametrize("short", ["parent", "draft", "target"])
def test_accepted_tokens_that_end_before_the_nodes(short):
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    a = dict(parent=[-1, 0, 1, -1, 0, 1], draft=[1] * 6, target=[1] * 6)
    a[short] = a[short][:5]
    out = [i32([99, 99]) for _ in range(3)]
    err = i32([0])
    L.check(L.la_tree_accept(i32([0, 3, 6]), i32(a["parent"]), 8, i32(a["draft"]), i32(a["target"]), i32([1, 1]), *out, err))
    torch.cuda.synchronize()
    assert int(err.item()) == L.DEVERR_CU_SEQLENS and [x.tolist() for x in out] == [[2, 99], [3, 99], [1, 99]]
