"""The bounded waits of the serving kernels, exercised without any fault: a test hook withholds
what one wait is for, so that the wait runs out after a short limit; the call must report
LA_DEVERR_TIMEOUT and return promptly, what does not depend on it is as ever, and so is the next
call."""
import time

import pytest
import torch

import serving_ref as R
from gated_deltanet_recurrent_la_b200 import lastate as L
from test_gpu_beam_slots import i32, slabs_of
from test_gpu_tree import device, run_tree

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _hooks_reset():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield
    L.la_debug_set_wait_limit_us(0)
    L.la_debug_withhold_step_tile(-1)


@pytest.mark.parametrize("lens", [[9, 3, 16, 1] * 12, [40, 64, 5, 33] * 12])  # one and two loads of the state
@pytest.mark.parametrize("rule,state_dtype,io_dtype", [("gated_delta", BF16, BF16), ("gated_delta", F32, F32), ("kda", BF16, BF16),
                                                       ("linear", F32, BF16)])
def test_tree_products_that_do_not_come(rule, state_dtype, io_dtype, lens):
    """More tiles than fit at once, so that tensor memory released by the one that gave up is used
    again while others run."""
    inp = R.tree_inputs(lens=lens, Hqk=8, Hv=16, dk=128, dv=128, rule=rule, state_dtype=state_dtype, io_dtype=io_dtype, seed=3)
    clean_o, clean_u, err = run_tree(device(inp))
    assert err == 0
    cu, d = inp["cu"].tolist(), device(inp)
    for b, h in ((0, 0), (2, 5), (5, 15)):
        L.la_debug_set_wait_limit_us(2000)
        L.la_debug_withhold_step_tile(b * 16 + h)
        t0 = time.perf_counter()
        o, u, err = run_tree(d)
        assert time.perf_counter() - t0 < 0.5
        assert err == L.DEVERR_TIMEOUT
        rows = slice(cu[b], cu[b + 1])
        assert torch.all(o[rows, h] == 7.0) and torch.all(u[rows, h] == 7.0)  # untouched
        o[rows, h], u[rows, h] = clean_o[rows, h], clean_u[rows, h]
        assert torch.equal(o, clean_o) and torch.equal(u, clean_u)
        o, u, err = run_tree(d)  # the hook is one-shot
        assert err == 0 and torch.equal(o, clean_o) and torch.equal(u, clean_u)


def test_tree_hooks_are_inert_when_not_reached():
    inp = R.tree_inputs(lens=[9, 20], Hqk=2, Hv=4, dk=64, dv=64, rule="gated_delta", state_dtype=BF16, io_dtype=BF16, seed=4)
    clean = run_tree(device(inp))
    L.la_debug_set_wait_limit_us(2000)
    L.la_debug_withhold_step_tile(8)  # tiles 0 .. 7
    again = run_tree(device(inp))
    assert again[2] == 0 and torch.equal(again[0], clean[0]) and torch.equal(again[1], clean[1])


def copied(host, dev, src, dst):
    return all(torch.equal(t[dst], h[src]) for h, t in zip(host, dev))


@pytest.mark.parametrize("piece", [0, 1, 4, 9])  # within the first round of the buffers and behind it
def test_slot_copies_that_do_not_come(piece):
    """60 slots of 104 pieces of 16 KiB: 12 or more for each of the up to 160 x 3 copying warps."""
    n_slots, src = 130, list(range(0, 120, 2))
    host = [t.cuda() for t in slabs_of(n_slots, [1 << 20, 2304, 600000, 16384, 48], 7)]
    dst = [s + 1 for s in src]

    def fork():
        dev = [t.clone() for t in host]
        ref = i32([1 if s in src else 0 for s in range(n_slots)])
        new, err = i32([55] * len(src)), i32([0])
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        L.check(L.la_state_pool_fork(L.Slabs(dev), ref, i32(src), new, err))
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 0.5
        assert new.tolist() == dst
        return dev, int(err.item())

    dev, err = fork()
    assert err == 0 and copied(host, dev, src, dst)
    L.la_debug_set_wait_limit_us(2000)
    L.la_debug_withhold_step_tile(piece)
    dev, err = fork()
    assert err == L.DEVERR_TIMEOUT and not copied(host, dev, src, dst)
    for h, t in zip(host, dev):  # every byte as it was or that of the slot's source
        assert torch.equal(t[src], h[src]) and torch.equal(t[120:], h[120:])
        assert torch.all((t[dst] == h[src]) | (t[dst] == h[dst]))
    dev, err = fork()  # the hook is one-shot
    assert err == 0 and copied(host, dev, src, dst)
