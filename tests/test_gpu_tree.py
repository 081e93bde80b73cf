"""Drafted token trees on the GPU (la_state_tree, la_tree_accept, la_state_tree_commit) against
the recurrence written out in 64 bits on explicit states.

Tolerances, from the arithmetic: FP32 sums err by at most tree_steps() times the magnitude bound
of the same recurrence on absolute values; a BF16 output adds one rounding (2^-8 of the value);
BF16 q, k, v may be multiplied on the tensor cores with the FP32 factors split into two BF16
terms each (a residue below 2^-16 of the magnitude, outputs only)."""
import numpy as np
import pytest
import torch

import serving_ref as R
from gated_deltanet_recurrent_la_b200 import lastate as L

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    L.lib()


def device(inp):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in inp.items()}


def run_tree(d, pool=None, want_u=True, max_nodes=None, guard=64):
    """o, u, error word; guard elements behind and before o and u must stay."""
    n = d["T"] * d["Hv"] * d["dv"]
    ob = torch.full((n + 2 * guard,), 7.0, dtype=d["q"].dtype, device="cuda")
    ub = torch.full((n + 2 * guard,), 7.0, device="cuda")
    o, u = (x[guard:guard + n].view(d["T"], d["Hv"], d["dv"]) for x in (ob, ub))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool = L.Pool(d["pool"], d["Hqk"]) if pool is None else pool
    L.check(L.la_state_tree(d["rule"], pool, d["read"], d["cu"], d["parent"], d["n"] if max_nodes is None else max_nodes,
                            d["q"], d["k"], d["v"], d["g"] if R.uses_gate(d["rule"]) else None,
                            d["beta"] if R.uses_beta(d["rule"]) else None, d["scale"], o, u if want_u else None, err))
    torch.cuda.synchronize()
    for x in (ob, ub):
        assert torch.all(x[:guard] == 7.0) and torch.all(x[guard + n:] == 7.0), "guard band overwritten"
    if not want_u:
        assert torch.all(ub == 7.0)
    return o.cpu(), u.cpu(), int(err.item())


def within(got, ref, mag, rel_mag, out_dtype, what):
    got, tol = got.double(), rel_mag * mag + (2.0 ** -8 * ref.abs() if out_dtype == BF16 else 0.0)
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - tol
    assert float(over.max()) <= 1e-30, f"{what}: {float(over.max()):.3e} over the bound"


def check_tree(inp, states=None, pool=None):
    o_ref, u_ref, mo, mu, depth = R.tree_ref(inp, inp["pool"] if states is None else states)
    o, u, err = run_tree(device(inp), pool)
    assert err == 0
    steps = R.tree_steps(depth, inp["dk"])
    within(u, u_ref, mu, steps, F32, "u")
    within(o, o_ref, mo, steps + (2.0 ** -16 if o.dtype == BF16 else 0.0), o.dtype, "o")
    return o, u


@pytest.mark.parametrize("state_dtype", [F32, BF16])
@pytest.mark.parametrize("io_dtype", [F32, BF16])
@pytest.mark.parametrize("rule", R.RULES)
@pytest.mark.parametrize("dk,dv", [(16, 16), (64, 64), (128, 64), (128, 128)])
def test_tree_every_rule_shape_and_type(dk, dv, rule, io_dtype, state_dtype):
    check_tree(R.tree_inputs(lens=[1, 0, 7, 16, 17, 33], Hqk=2, Hv=4, dk=dk, dv=dv, rule=rule, state_dtype=state_dtype,
                             io_dtype=io_dtype, seed=dk + dv))


@pytest.mark.parametrize("shape", ["chain", "star", "tree"])
@pytest.mark.parametrize("rule", ["gated_delta", "kda", "gated"])
@pytest.mark.parametrize("io_dtype,state_dtype", [(BF16, BF16), (F32, F32), (BF16, F32)])
def test_tree_largest(shape, rule, io_dtype, state_dtype):
    check_tree(R.tree_inputs(lens=[64, 63, 49, 48], Hqk=1, Hv=3, dk=128, dv=128, rule=rule, state_dtype=state_dtype,
                             io_dtype=io_dtype, seed=5, shape=shape))


@pytest.mark.parametrize("n", [1, 2, 8, 9, 15, 16, 24, 31, 32, 40, 48, 57, 64])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64)])
def test_tree_sizes(n, dk, dv):
    check_tree(R.tree_inputs(lens=[n, max(1, n // 2), n], Hqk=2, Hv=2, dk=dk, dv=dv, rule="gated_delta", state_dtype=BF16,
                             io_dtype=BF16, seed=n))


@pytest.mark.parametrize("rule", ["gated", "gated_delta", "kda"])
@pytest.mark.parametrize("io_dtype", [F32, BF16])
def test_tree_gates_of_either_sign_and_zero(rule, io_dtype):
    check_tree(R.tree_inputs(lens=[12, 20, 5], Hqk=2, Hv=4, dk=128, dv=128, rule=rule, state_dtype=BF16, io_dtype=io_dtype,
                             seed=9, wide=True))


@pytest.mark.parametrize("Hqk,Hv,B", [(1, 1, 1), (1, 8, 3), (16, 32, 2), (4, 4, 40)])
def test_tree_head_layouts_and_batches(Hqk, Hv, B):
    check_tree(R.tree_inputs(lens=[(3 * b) % 11 for b in range(B - 1)] + [6], Hqk=Hqk, Hv=Hv, dk=128, dv=128,
                             rule="gated_delta", state_dtype=BF16, io_dtype=BF16, seed=B))


def test_tree_of_one_node_is_the_decode_step():
    inp = R.tree_inputs(lens=[1] * 5, Hqk=2, Hv=4, dk=128, dv=128, rule="gated_delta", state_dtype=F32, io_dtype=F32, seed=3)
    o, _, _ = run_tree(device(inp))
    d = device(inp)
    new = torch.zeros(5, 4, 128, 128, device="cuda")
    o2 = torch.zeros(5, 4, 128, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.check(L.la_state_step("gated_delta", L.Pool(d["pool"], 2), d["read"], L.Pool(new, 2), None, d["q"], d["k"], d["v"],
                            d["g"], d["beta"], inp["scale"], o2, err))
    torch.cuda.synchronize()
    _, _, mo, _, _ = R.tree_ref(inp, inp["pool"])
    assert float(((o - o2.cpu()).abs() - 2 * R.tree_steps(1, 128) * mo).max()) <= 0


def test_tree_same_state_read_twice_and_no_slot_array():
    inp = R.tree_inputs(lens=[4, 9, 4], Hqk=1, Hv=2, dk=64, dv=64, rule="delta", state_dtype=BF16, io_dtype=BF16, seed=4)
    inp["read"] = torch.tensor([2, 2, 0], dtype=torch.int32)
    check_tree(inp)
    d = device(inp)
    d["read"] = None
    o, _, err = run_tree(d)
    inp["read"] = torch.tensor([0, 1, 2], dtype=torch.int32)
    o2, _, _ = run_tree(device(inp))
    assert err == 0 and torch.equal(o, o2)


def test_tree_without_write_vectors():
    inp = R.tree_inputs(lens=[5, 30], Hqk=1, Hv=2, dk=128, dv=128, rule="gated_delta", state_dtype=BF16, io_dtype=BF16, seed=6)
    o, _, _ = run_tree(device(inp), want_u=True)
    o2, _, err = run_tree(device(inp), want_u=False)
    assert err == 0 and torch.equal(o, o2)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["v", "q", "beta", "k"])
@pytest.mark.parametrize("io_dtype", [F32, BF16])
@pytest.mark.parametrize("rule", ["gated_delta", "kda"])
def test_tree_nonfinite_branch_stays_in_its_branch(value, where, io_dtype, rule):
    """A non-finite value of one node reaches that node and those below it, no other."""
    inp = R.tree_inputs(lens=[20, 20], Hqk=1, Hv=2, dk=128, dv=128, rule=rule, state_dtype=BF16, io_dtype=io_dtype, seed=8)
    parent = inp["parent"].tolist()
    bad = next(t for t in range(1, 20) if any(parent[c] == t for c in range(20)) and parent[t] >= 0)
    clean, cu_, err = run_tree(device(inp))
    broken = dict(inp)
    broken[where] = inp[where].clone()
    broken[where][bad] = value
    got, gu, err = run_tree(device(broken))
    assert err == 0
    below = {bad} if where != "q" else set()
    for t in range(20):
        if parent[t] in below:
            below.add(t)
    below |= {bad}
    for t in range(40):
        if t not in below:
            assert torch.equal(got[t], clean[t]) and torch.equal(gu[t], cu_[t]), t
    assert not torch.isfinite(got[bad].float()).all()


def test_tree_infinite_state_of_another_sequence():
    inp = R.tree_inputs(lens=[6, 6], Hqk=1, Hv=1, dk=128, dv=128, rule="gated_delta", state_dtype=BF16, io_dtype=BF16, seed=2)
    clean, _, _ = run_tree(device(inp))
    inp["pool"][int(inp["read"][0])] = float("inf")
    got, _, err = run_tree(device(inp))
    assert err == 0 and torch.equal(got[6:], clean[6:])


def q8_pool(inp, seed=1):
    """The inputs' states in a q8 pool, its decoded values [slots, Hv, dk, dv], and the pool."""
    slots, Hv, dk, dv = inp["pool"].shape
    n_hp = dk // 8
    rng = np.random.RandomState(seed)
    words = np.zeros((Hv, dk // 32), np.uint32)
    for h in range(Hv):
        for c in rng.permutation(dk)[:n_hp]:
            words[h, c // 32] |= np.uint32(1 << (c % 32))
    mask = torch.tensor(words.view(np.int32)).cuda()
    data = torch.zeros(slots, Hv, L.q8_tile_bytes(dk, dv, n_hp), dtype=torch.uint8, device="cuda")
    pool = L.Pool.q8(data, inp["Hqk"], dk, dv, n_hp, mask)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    every = torch.arange(slots, dtype=torch.int32, device="cuda")
    L.check(L.la_state_pool_encode(pool, every, inp["pool"].float().cuda(), err))
    return pool, q8_values(pool, every), mask


def q8_values(pool, slots):
    dk, dv = pool.struct.shape.d_k, pool.struct.shape.d_v
    out = torch.zeros(slots.numel(), pool.struct.shape.n_v_heads, dk, dv, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.check(L.la_state_pool_decode(pool, slots, out, err))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out.cpu()


@pytest.mark.parametrize("rule", ["gated_delta", "kda", "linear"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("io_dtype", [F32, BF16])
def test_tree_and_commit_on_q8_pools(rule, dk, dv, io_dtype):
    inp = R.tree_inputs(lens=[3, 20, 1, 6], Hqk=2, Hv=4, dk=dk, dv=dv, rule=rule, state_dtype=F32, io_dtype=io_dtype, seed=7)
    pool, values, mask = q8_pool(inp)
    _, u = check_tree(inp, states=values, pool=pool)
    leaf = torch.tensor([2, 13, -1, 5], dtype=torch.int32)
    dst_t = torch.full((4,) + tuple(pool.tensor.shape[1:]), 9, dtype=torch.uint8, device="cuda")
    dst = L.Pool.q8(dst_t, inp["Hqk"], dk, dv, dk // 8, mask)
    err = commit(device(inp), pool, dst, None, leaf, u)
    assert err == 0
    ref, mag = R.commit_ref(inp, values, leaf, u)
    got = q8_values(dst, torch.arange(4, dtype=torch.int32, device="cuda")).double()
    # a code is off by half a step of its 32-column group (absmax / 127, itself within 2^-22), a BF16 row by 2^-8
    group = ref.abs().reshape(4, 4, dk, dv // 32, 32).amax(-1, keepdim=True).expand(4, 4, dk, dv // 32, 32).reshape(ref.shape)
    assert float(((got - ref).abs() - (group * (0.5 / 127 * (1 + 2.0 ** -10)) + 64 * 2.0 ** -24 * mag)).max()) <= 0
    assert torch.equal(dst_t[2], pool.tensor[int(inp["read"][2])])  # nothing accepted: the codes as they are


def commit(d, src, dst, write, leaf, u, max_nodes=None):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.check(L.la_state_tree_commit(d["rule"], src, d["read"], dst, write, d["cu"], d["parent"], leaf.cuda(),
                                   d["n"] if max_nodes is None else max_nodes, d["k"],
                                   d["g"] if R.uses_gate(d["rule"]) else None, u.cuda(), err))
    torch.cuda.synchronize()
    return int(err.item())


@pytest.mark.parametrize("state_dtype", [F32, BF16])
@pytest.mark.parametrize("io_dtype", [F32, BF16])
@pytest.mark.parametrize("rule", R.RULES)
@pytest.mark.parametrize("dk,dv", [(16, 16), (64, 64), (128, 64), (128, 128)])
def test_commit_every_rule_shape_and_type(dk, dv, rule, io_dtype, state_dtype):
    lens = [1, 0, 7, 16, 33, 64]
    inp = R.tree_inputs(lens=lens, Hqk=2, Hv=4, dk=dk, dv=dv, rule=rule, state_dtype=state_dtype, io_dtype=io_dtype,
                        seed=dk * 3 + dv, wide=rule != "gated_delta", shape="chain" if rule == "delta" else "tree")
    gen = torch.Generator().manual_seed(1)
    u = torch.randn(inp["T"], 4, dv, generator=gen)
    leaf = torch.tensor([0, -1, 6, -1, 32, 63], dtype=torch.int32)
    ref, mag = R.commit_ref(inp, inp["pool"], leaf, u)
    d = device(inp)
    dst_t = torch.full((9, 4, dk, dv), 3.0, dtype=state_dtype, device="cuda")
    write = torch.tensor([7, 0, 3, 8, 1, 5], dtype=torch.int32, device="cuda")
    assert commit(d, L.Pool(d["pool"], 2), L.Pool(dst_t, 2), write, leaf, u) == 0
    got = dst_t.cpu()[write.cpu().long()]
    # a path of at most 64 nodes: so many products and additions
    within(got, ref, mag, 200 * 2.0 ** -24, state_dtype, "state")
    assert torch.equal(got[3], inp["pool"][int(inp["read"][3])]) and torch.equal(got[1], inp["pool"][int(inp["read"][1])])
    rest = [s for s in range(9) if s not in write.tolist()]
    assert torch.all(dst_t[rest] == 3.0) and torch.equal(d["pool"].cpu(), inp["pool"])


def test_commit_in_place():
    inp = R.tree_inputs(lens=[10, 4, 20], Hqk=1, Hv=2, dk=128, dv=128, rule="kda", state_dtype=BF16, io_dtype=BF16, seed=21)
    u = torch.randn(inp["T"], 2, 128, generator=torch.Generator().manual_seed(2))
    leaf = torch.tensor([9, -1, 17], dtype=torch.int32)
    ref, mag = R.commit_ref(inp, inp["pool"], leaf, u)
    d = device(inp)
    pool = L.Pool(d["pool"], 1)
    assert commit(d, pool, pool, d["read"], leaf, u) == 0
    got = d["pool"].cpu()
    within(got[inp["read"].long()], ref, mag, 200 * 2.0 ** -24, BF16, "state")
    other = [s for s in range(got.shape[0]) if s not in inp["read"].tolist()]
    assert torch.equal(got[other], inp["pool"][other])


def test_commit_does_not_read_other_branches():
    """u and k off the path may hold anything."""
    inp = R.tree_inputs(lens=[30], Hqk=1, Hv=1, dk=64, dv=64, rule="gated", state_dtype=F32, io_dtype=F32, seed=22)
    u = torch.randn(30, 1, 64, generator=torch.Generator().manual_seed(3))
    leaf = torch.tensor([20], dtype=torch.int32)
    path, t = set(), 20
    while t >= 0:
        path.add(t)
        t = int(inp["parent"][t])
    for t in range(30):
        if t not in path:
            u[t], inp["k"][t], inp["g"][t] = float("nan"), float("inf"), float("nan")
    ref, mag = R.commit_ref(inp, inp["pool"], leaf, u)
    d = device(inp)
    dst = torch.zeros(1, 1, 64, 64, device="cuda")
    assert commit(d, L.Pool(d["pool"], 1), L.Pool(dst, 1), None, leaf, u) == 0
    within(dst.cpu(), ref, mag, 200 * 2.0 ** -24, F32, "state")


@pytest.mark.parametrize("seed", range(6))
def test_accept(seed):
    rng = np.random.RandomState(seed)
    lens = [0, 1, 64, 33, 32, 5] + [int(rng.randint(0, 65)) for _ in range(40)]
    cu = np.concatenate([[0], np.cumsum(lens)])
    parent = [p for n in lens for p in R.random_parents(rng, n, "chain" if seed == 1 else "tree")]
    vocab = 2 if seed < 3 else 4  # few tokens: siblings with the same one
    T = len(parent)
    draft, target, root = rng.randint(0, vocab, T), rng.randint(0, vocab, T), rng.randint(0, vocab, len(lens))
    want = R.accept_ref(cu.tolist(), parent, draft, target, root)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    leaf, count, nxt, err = (i32(np.full(len(lens), 99)) for _ in range(4))
    err = i32([0])
    L.check(L.la_tree_accept(i32(cu), i32(parent), 64, i32(draft), i32(target), i32(root), leaf, count, nxt, err))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert [leaf.tolist(), count.tolist(), nxt.tolist()] == [list(x) for x in want]


def test_device_errors_skip_the_sequence():
    inp = R.tree_inputs(lens=[5, 6, 7, 8], Hqk=1, Hv=2, dk=128, dv=128, rule="gated_delta", state_dtype=BF16, io_dtype=BF16,
                        seed=31)
    clean, _, _ = run_tree(device(inp))
    cu = inp["cu"].tolist()

    def case(bits, seq, **change):
        d = device({**inp, **change})
        o, u, err = run_tree(d, max_nodes=change.get("max_nodes"))
        assert err == bits
        for b in range(4):
            rows = slice(cu[b], cu[b + 1])
            if b in seq:
                assert torch.all(o[rows] == 7.0) and torch.all(u[rows] == 7.0)
            else:
                assert torch.equal(o[rows], clean[rows])

    read = inp["read"].clone()
    read[1] = 9
    case(L.DEVERR_READ_SLOT, [1], read=read)
    read[1] = -1
    case(L.DEVERR_READ_SLOT, [1], read=read)
    for bad in (5, 7, -2):
        parent = inp["parent"].clone()
        parent[cu[2] + 5] = bad
        case(L.DEVERR_TREE, [2], parent=parent)
    case(L.DEVERR_TREE, [3], max_nodes=7)
    cub = inp["cu"].clone()
    cub[4] = 99
    case(L.DEVERR_CU_SEQLENS, [3], cu=cub)

    d = device(inp)
    u = torch.randn(inp["T"], 2, 128)
    leaf = torch.tensor([4, 6, -2, 7], dtype=torch.int32)  # sequence 1 has 6 nodes
    dst = torch.full((4, 2, 128, 128), 3.0, dtype=BF16, device="cuda")
    src = L.Pool(d["pool"], 1)
    assert commit(d, src, L.Pool(dst, 1), None, leaf, u) == L.DEVERR_TREE
    assert torch.all(dst[1] == 3.0) and torch.all(dst[2] == 3.0) and not torch.all(dst[0] == 3.0)
    write = torch.tensor([0, 4, 2, 3], dtype=torch.int32, device="cuda")
    leaf = torch.tensor([4, 5, 6, 7], dtype=torch.int32)
    dst.fill_(3.0)
    assert commit(d, src, L.Pool(dst, 1), write, leaf, u) == L.DEVERR_WRITE_SLOT
    assert torch.all(dst[1] == 3.0)

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    parent = inp["parent"].clone()
    parent[cu[1] + 2] = 3
    out = [i32([99] * 4) for _ in range(3)]
    err = i32([0])
    zeros = torch.zeros(inp["T"], dtype=torch.int32, device="cuda")
    L.check(L.la_tree_accept(d["cu"], parent.cuda(), 8, zeros, zeros, i32([1] * 4), *out, err))
    assert int(err.item()) == L.DEVERR_TREE
    assert [x.tolist() for x in out] == [[-1, 99, -1, -1], [0, 99, 0, 0], [1, 99, 1, 1]]


def test_captured_and_replayed_on_a_side_stream():
    """Verification, acceptance and commit as one captured round, replayed on new inputs."""
    a = R.tree_inputs(lens=[8, 12, 3], Hqk=2, Hv=4, dk=128, dv=128, rule="gated_delta", state_dtype=BF16, io_dtype=BF16, seed=41)
    b = R.tree_inputs(lens=[12, 1, 10], Hqk=2, Hv=4, dk=128, dv=128, rule="gated_delta", state_dtype=BF16, io_dtype=BF16, seed=42)
    assert a["T"] == b["T"]
    d = device(a)
    pool = L.Pool(d["pool"], 2)
    T = a["T"]
    o, u = torch.zeros(T, 4, 128, dtype=BF16, device="cuda"), torch.zeros(T, 4, 128, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    draft, target, root = i32([1] * T), i32([1] * T), i32([1] * 3)
    leaf, count, nxt, err = i32([0] * 3), i32([0] * 3), i32([0] * 3), i32([0])

    def round_():
        L.check(L.la_state_tree("gated_delta", pool, d["read"], d["cu"], d["parent"], 12, d["q"], d["k"], d["v"], d["g"],
                                d["beta"], 0.75, o, u, err))
        L.check(L.la_tree_accept(d["cu"], d["parent"], 12, draft, target, root, leaf, count, nxt, err))
        L.check(L.la_state_tree_commit("gated_delta", pool, d["read"], pool, d["read"], d["cu"], d["parent"], leaf, 12,
                                       d["k"], d["g"], u, err))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        round_()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            round_()
    for inp in (b, a):
        for name in ("pool", "read", "cu", "parent", "q", "k", "v", "g", "beta"):
            d[name].copy_(inp[name])
        graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        o_ref, u_ref, mo, mu, depth = R.tree_ref(inp, inp["pool"])
        within(o.cpu(), o_ref, mo, R.tree_steps(depth, 128) + 2.0 ** -16, BF16, "o")
        want = R.accept_ref(inp["cu"].tolist(), inp["parent"].tolist(), [1] * T, [1] * T, [1] * 3)
        assert [leaf.tolist(), count.tolist(), nxt.tolist()] == [list(x) for x in want]
        S, mag = R.commit_ref(inp, inp["pool"], leaf.cpu(), u.cpu())
        within(d["pool"].cpu()[inp["read"].long()], S, mag, 200 * 2.0 ** -24, BF16, "state")


def test_repeated_calls_give_the_same_bits():
    inp = R.tree_inputs(lens=[40, 64, 7], Hqk=2, Hv=4, dk=128, dv=128, rule="gated_delta", state_dtype=BF16, io_dtype=BF16, seed=51)
    d = device(inp)
    first = run_tree(d)
    for _ in range(3):
        again = run_tree(d)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
