"""The serving operators where their kernels change form: FP32 operands on the tensor cores, rows
whose best values crowd one part of the selection, masks of the type's lowest value, batches of
slots beyond one CTA's list, captured selection and reordering."""
import numpy as np
import pytest
import torch

import serving_ref as R
from gated_deltanet_recurrent_la_b200 import lastate as L
from test_gpu_beam_slots import beam_inputs, check_select, i32, select, slabs_of
from test_gpu_tree import device, run_tree

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    L.lib()


def recurrence_fp32(inp):
    """o and u by elementary FP32 operations on explicit states."""
    ratio = inp["Hv"] // inp["Hqk"]
    q, k = (inp[x].float().repeat_interleave(ratio, 1) for x in ("q", "k"))
    v, g, beta = inp["v"].float(), inp["g"], inp["beta"]
    o, u = torch.zeros_like(v), torch.zeros_like(v)
    cu, parent = inp["cu"].tolist(), inp["parent"].tolist()
    for b in range(inp["B"]):
        S = {-1: inp["pool"][int(inp["read"][b])].float()}
        for t in range(cu[b], cu[b + 1]):
            s = R.decayed(inp["rule"], S[parent[t]], g[t])
            u[t] = v[t] if not R.uses_beta(inp["rule"]) else beta[t][:, None] * (v[t] - (s * k[t][:, :, None]).sum(1))
            S[t - cu[b]] = s + k[t][:, :, None] * u[t][:, None, :]
            o[t] = inp["scale"] * (S[t - cu[b]] * q[t][:, :, None]).sum(1)
    return o, u


@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("n,shape", [(64, "chain"), (57, "tree"), (20, "tree"), (9, "chain")])
@pytest.mark.parametrize("rule,state_dtype", [("gated_delta", F32), ("kda", F32), ("delta", BF16), ("linear", F32)])
def test_fp32_operands_lose_nothing(rule, state_dtype, n, shape, dk, dv):
    """The error against 64 bits, over all outputs, is at most three times that of elementary FP32:
    both are sums of roundings of 2^-24 of the partial sums, d_k / 16 truncations and the path's
    additions here, d_k additions and the path's there, so that the ratio is near one."""
    inp = R.tree_inputs(lens=[n, max(1, n - 3)], Hqk=1, Hv=2, dk=dk, dv=dv, rule=rule, state_dtype=state_dtype, io_dtype=F32,
                        seed=n, shape=shape)
    o_ref, u_ref, _, _, _ = R.tree_ref(inp, inp["pool"])
    o, u, err = run_tree(device(inp))
    assert err == 0
    o32, u32 = recurrence_fp32(inp)
    for got, plain, ref in ((o, o32, o_ref), (u, u32, u_ref)):
        mine, theirs = (float((x.double() - ref).norm() / ref.norm()) for x in (got, plain))
        assert mine <= 3 * theirs + 2.0 ** -30, (mine, theirs)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_select_best_values_in_one_stride(dtype):
    """All large values lie in pieces a power of two apart, more of them than a list holds."""
    V, E = 1 << 21, 4 if dtype == F32 else 8
    gen = torch.Generator().manual_seed(1)
    logits = torch.randn(1, 1, V, generator=gen)
    crowd = (torch.arange(V) // E) % 128 == 7
    logits[0, 0, crowd] += 60.0
    x = logits.to(dtype)
    cum = torch.tensor([[-0.25]])
    for n_out in (1, 24):
        par, tok, sc, _, _ = R.beam_ref(x, cum.numpy(), None, -1, n_out)
        p, t, s, _ = select(x, cum, None, -1, n_out)
        np.testing.assert_array_equal(t, tok)
        assert np.all(p == 0) and np.all(np.abs(s - sc) <= 2.0 ** -20 + 2.0 ** -23 * np.abs(sc))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [97, 9000])
def test_select_masks_of_the_lowest_value(dtype, V):
    """A mask of the type's lowest value leaves the other tokens their scores; a row of nothing
    else is a uniform one far down."""
    low = torch.finfo(dtype).min
    logits, cum = beam_inputs(3, 2, V, dtype, seed=V, masked=0.0)
    logits[:, :, V // 3:] = low
    check_select(logits, cum, None, -1, 4)
    for rows in ((0,), (0, 1)):  # one beam, then every beam of the first sequence
        for i in rows:
            logits[0, i] = low
        x = logits.double().numpy()
        x = x - x.max(2, keepdims=True)  # before anything is added to 1e38
        want = cum.double().numpy()[..., None] + (x - np.log(np.exp(x).sum(2, keepdims=True)))
        p, t, s, _ = select(logits, cum, None, -1, 4)
        for b in range(3):
            best = np.lexsort((np.arange(2 * V), -want[b].reshape(-1)))[:4]
            np.testing.assert_array_equal(p[b], best // V)
            np.testing.assert_array_equal(t[b], best % V)
            w = want[b].reshape(-1)[best]
            assert np.all(np.abs(s[b] - w) <= 2.0 ** -20 + 2.0 ** -23 * np.abs(w))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_select_an_offset_of_all_logits_cancels(dtype):
    """Logits in a narrow band far from zero: differences keep their weight."""
    base = 4096.0 if dtype == F32 else 64.0
    gen = torch.Generator().manual_seed(3)
    logits = (base + torch.randint(-8, 9, (2, 3, 5000), generator=gen) * 0.5).to(dtype)
    cum = torch.tensor([[0.0, -0.31, -0.83]] * 2)
    par, tok, sc, _, _ = R.beam_ref(logits, cum.numpy(), None, -1, 6)
    p, t, s, _ = select(logits, cum, None, -1, 6)
    np.testing.assert_array_equal(t, tok)
    np.testing.assert_array_equal(p, par)
    assert np.all(np.abs(s - sc) <= 2.0 ** -20 + 2.0 ** -23 * np.abs(sc))


@pytest.mark.parametrize("B,K", [(70, 8), (7, 61), (300, 1)])
def test_reorder_of_many_sequences(B, K):
    """More pairs than one list of the copying CTAs holds."""
    rng = np.random.RandomState(B)
    n_slots = B * K + 1
    slots = rng.permutation(n_slots)[:B * K].reshape(B, K)
    parent = rng.randint(0, K, (B, K))
    host = slabs_of(n_slots, [48, 33 * 1024 + 16], 5)
    dev = [t.cuda() for t in host]
    new, err = i32(np.full((B, K), 55)), i32([0])
    L.check(L.la_state_pool_reorder(L.Slabs(dev), i32(slots), i32(parent), new, err))
    torch.cuda.synchronize()
    want, copies = R.reorder_ref(slots.tolist(), parent.tolist())
    assert int(err.item()) == 0 and new.tolist() == want
    for h, t in zip(host, dev):
        expect = h.clone()
        for s, d in copies:
            expect[d] = h[s]
        assert torch.equal(t.cpu(), expect)


def test_captured_selection_and_reordering():
    """One graph of a beam step, replayed on other logits; two graphs share the workspace."""
    B, K, V = 3, 4, 9000
    spec = [4096, 16400]
    logits = torch.zeros(B, K, V, device="cuda")
    cum = torch.zeros(B, K, device="cuda")
    slots = i32(np.arange(B * K).reshape(B, K))
    ws = torch.empty(L.la_beam_workspace_bytes(B, K, V, K), dtype=torch.uint8, device="cuda")
    err = i32([0])
    slabs = [t.cuda() for t in slabs_of(B * K, spec, 1)]
    handle = L.Slabs(slabs)
    outs = [[i32(np.full((B, K), 55)) for _ in range(4)] + [torch.zeros(B, K, device="cuda")] for _ in range(2)]

    def step(out):
        parent, token, fin, new, score = out
        L.check(L.la_beam_select(logits, cum, None, -1, parent, token, score, fin, ws))
        L.check(L.la_state_pool_reorder(handle, slots, parent, new, err))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        step(outs[0])
        side.synchronize()
        for out in outs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                step(out)
            graphs.append(g)
    for seed, (g, out) in enumerate(zip(graphs * 2, outs * 2)):
        host = slabs_of(B * K, spec, seed)
        for t, h in zip(slabs, host):
            t.copy_(h)
        x, c = beam_inputs(B, K, V, F32, seed=40 + seed)
        logits.copy_(x)
        cum.copy_(c)
        g.replay()
        torch.cuda.synchronize()
        par, tok, _, _, gap = R.beam_ref(x, c.numpy(), None, -1, K)
        assert gap > 1e-5
        np.testing.assert_array_equal(out[0].cpu().numpy(), par)
        np.testing.assert_array_equal(out[1].cpu().numpy(), tok)
        want, copies = R.reorder_ref(slots.tolist(), par.tolist())
        assert out[3].tolist() == want and int(err.item()) == 0
        for t, h in zip(slabs, host):
            expect = h.clone()
            for s, d in copies:
                expect[d] = h[s]
            assert torch.equal(t.cpu(), expect)


def test_two_streams_verify_at_once():
    """Trees of different sizes and types on two streams share the SMs' tensor memory."""
    cases = [R.tree_inputs(lens=[64] * 24, Hqk=2, Hv=8, dk=128, dv=128, rule="gated_delta", state_dtype=BF16, io_dtype=BF16, seed=1),
             R.tree_inputs(lens=[30] * 40, Hqk=2, Hv=8, dk=128, dv=128, rule="gated_delta", state_dtype=F32, io_dtype=F32, seed=2)]
    alone = [run_tree(device(c)) for c in cases]
    ds, streams, outs = [device(c) for c in cases], [torch.cuda.Stream() for _ in cases], []
    torch.cuda.synchronize()
    for rounds in range(3):
        for d, s in zip(ds, streams):
            o = torch.zeros(d["T"], d["Hv"], 128, dtype=d["q"].dtype, device="cuda")
            u = torch.zeros(d["T"], d["Hv"], 128, device="cuda")
            err = i32([0])
            s.wait_stream(torch.cuda.current_stream())
            L.check(L.la_state_tree(d["rule"], L.Pool(d["pool"], d["Hqk"]), d["read"], d["cu"], d["parent"], d["n"], d["q"],
                                    d["k"], d["v"], d["g"], d["beta"], d["scale"], o, u, err, stream=s))
            outs.append((o, u, err))
    torch.cuda.synchronize()
    for i, (o, u, err) in enumerate(outs):
        assert int(err.item()) == 0
        assert torch.equal(o.cpu(), alone[i % 2][0]) and torch.equal(u.cpu(), alone[i % 2][1])
