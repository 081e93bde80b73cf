"""Beam selection and slot bookkeeping on the GPU (la_beam_select, la_state_pool_reorder, _alloc,
_share, _free, _fork, _compact, _remap) against plain implementations, whole numbers and copies
exactly.  Scores: logsumexp from FP32 exponentials (2 units in the last place each) and FP32
partial sums is within 2^-20, the stored score one rounding (2^-24 of it) more."""
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


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def select(logits, cum, finished, eos, n_out, logits_dev=None):
    B, K, V = logits.shape
    x = logits.cuda() if logits_dev is None else logits_dev
    parent, token, fin = (torch.full((B, n_out), 77, dtype=torch.int32, device="cuda") for _ in range(3))
    score = torch.full((B, n_out), 77.0, device="cuda")
    ws = torch.empty(L.la_beam_workspace_bytes(B, K, V, n_out), dtype=torch.uint8, device="cuda")
    L.check(L.la_beam_select(x, cum.cuda(), None if finished is None else finished.cuda(), eos, parent, token, score, fin, ws))
    torch.cuda.synchronize()
    return parent.cpu().numpy(), token.cpu().numpy(), score.cpu().numpy(), fin.cpu().numpy()


def check_select(logits, cum, finished, eos, n_out, logits_dev=None):
    par, tok, sc, fin, gap = R.beam_ref(logits, cum.numpy(), None if finished is None else finished.numpy(), eos, n_out)
    assert gap > 1e-5, "the inputs' own scores are too close to tell apart: another seed"
    p, t, s, f = select(logits, cum, finished, eos, n_out, logits_dev)
    np.testing.assert_array_equal(p, par)
    np.testing.assert_array_equal(t, tok)
    np.testing.assert_array_equal(f, fin)
    fine = np.isfinite(sc)
    np.testing.assert_array_equal(s[~fine], sc[~fine])
    assert np.all(np.abs(s[fine] - sc[fine]) <= 2.0 ** -20 + 2.0 ** -23 * np.abs(sc[fine]))


def beam_inputs(B, K, V, dtype, seed, masked=0.1):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(B, K, V, generator=gen) * 3
    x[torch.rand(B, K, V, generator=gen) < masked] = -float("inf")
    cum = -torch.rand(B, K, generator=gen).cumsum(1) * 2
    return x.to(dtype), cum


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,K,V,n_out", [(1, 1, 1, 1), (1, 1, 2, 2), (2, 3, 5, 4), (3, 2, 7, 14), (1, 4, 31, 8), (2, 4, 1000, 4),
                                         (5, 8, 1025, 16), (2, 5, 4099, 10), (1, 3, 32000, 6), (2, 2, 50257, 2),
                                         (1, 16, 8191, 16), (1, 64, 300, 64), (1, 1, 131072, 64), (1, 2, 9000, 33)])
def test_select(B, K, V, n_out, dtype):
    logits, cum = beam_inputs(B, K, V, dtype, seed=B * 1000 + K * 100 + V % 97)
    check_select(logits, cum, None, -1, n_out)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_select_first_step_finished_and_masked_rows(dtype):
    logits, cum = beam_inputs(6, 4, 700, dtype, seed=5)
    cum[0, 1:] = -float("inf")          # one live beam
    cum[1] = -float("inf")              # none: every candidate -inf, the lowest ones
    logits[2, 0] = -float("inf")        # a beam whose mask leaves nothing
    logits[3] = -float("inf")           # ... every beam
    fin = torch.zeros(6, 4, dtype=torch.int32)
    fin[2, 3] = fin[4, 0] = fin[4, 1] = 1
    fin[5] = 1                          # every beam finished: four continuations, then -inf
    cum[0, 2], fin[0, 2] = -float("inf"), 1
    check_select(logits, cum, fin, 3, 4)
    check_select(logits, cum, fin, 699, 9)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [64, 5000, 33000])
def test_select_ties_go_to_the_lowest(dtype, V):
    gen = torch.Generator().manual_seed(V)
    logits = torch.randint(-3, 3, (3, 3, V), generator=gen).to(dtype)   # few values: every best is shared
    logits[1] = 0.0                                                     # all equal
    logits[2, :, 1::2] = -0.0
    logits[2, :, ::2] = 0.0                                             # -0 equals +0
    cum = torch.tensor([[0.0, -0.125, -0.375]] * 3)
    cum[1] = torch.tensor([0.0, -0.25, -0.5])
    par, tok, sc, _, _ = R.beam_ref(logits, cum.numpy(), None, -1, 12)
    p, t, s, _ = select(logits, cum, None, -1, 12)
    np.testing.assert_array_equal(p, par)
    np.testing.assert_array_equal(t, tok)
    assert np.all(np.abs(s - sc) <= 2.0 ** -20 + 2.0 ** -23 * np.abs(sc))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_select_best_values_bunched_together(dtype):
    """Descending and ascending rows, and all of the best in neighbouring places."""
    V = 20000
    logits = torch.zeros(1, 3, V)
    logits[0, 0] = -torch.arange(V) * 0.5
    logits[0, 1] = torch.arange(V) * 0.5 - 0.5 * V
    logits[0, 2, 7000:7064] = 40.0 + torch.arange(64)
    cum = torch.tensor([[-1.1, -0.3, -2.7]])
    x = logits.to(dtype)
    for n_out in (1, 16, 64):
        par, tok, sc, _, _ = R.beam_ref(x, cum.numpy(), None, -1, n_out)
        p, t, s, _ = select(x, cum, None, -1, n_out)
        np.testing.assert_array_equal(p, par)
        np.testing.assert_array_equal(t, tok)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_select_infinities_and_nan(dtype):
    logits, cum = beam_inputs(2, 2, 300, dtype, seed=11)
    logits[0, 0, 5], logits[0, 1, 7] = float("nan"), -float("inf")
    logits[1, 0, 9] = float("nan")
    check_select(logits, cum, None, -1, 5)
    logits[0, 0, 100] = float("inf")  # as the largest float: all the others have no weight beside it
    p, t, s, _ = select(logits, cum, None, -1, 5)
    assert (0, 100) in list(zip(p[0], t[0])) and np.isfinite(s[0][list(t[0]).index(100)])
    par, tok, _, _, _ = R.beam_ref(logits[1:], cum[1:].numpy(), None, -1, 5)
    np.testing.assert_array_equal(t[1], tok[0])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset,extra", [(0, 0), (1, 3), (3, 13), (8, 8), (5, 0)])
def test_select_strided_and_unaligned_rows(dtype, offset, extra):
    """Rows of a padded vocabulary, starting anywhere; what lies between them is not looked at."""
    B, K, V = 2, 3, 4001
    logits, cum = beam_inputs(B, K, V, dtype, seed=offset + 17)
    flat = torch.full((offset + B * K * (V + extra) + 64,), 1e9, dtype=dtype, device="cuda")
    rows = flat[offset:offset + B * K * (V + extra)].view(B, K, V + extra)
    view = rows[:, :, :V]
    view.copy_(logits)
    check_select(logits, cum, None, -1, 6, logits_dev=view)


def slabs_of(n_slots, spec, seed):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randint(-128, 127, (n_slots, size), dtype=torch.int8, generator=gen) for size in spec]


SPECS = [[16], [48, 16384], [4096, 16400, 32], [65536, 2304, 65536, 2304]]


@pytest.mark.parametrize("spec", SPECS)
@pytest.mark.parametrize("B,K", [(1, 1), (1, 4), (3, 8), (2, 33), (1, 64), (40, 2)])
def test_reorder(B, K, spec):
    rng = np.random.RandomState(B + K)
    n_slots = B * K + 3
    slots = rng.permutation(n_slots)[:B * K].reshape(B, K)
    parent = rng.randint(0, K, (B, K))
    parent[-1] = rng.permutation(K)  # a permutation: nothing is copied
    host = slabs_of(n_slots, spec, 1)
    dev = [t.cuda() for t in host]
    new, err = torch.full((B, K), 55, dtype=torch.int32, device="cuda"), i32([0])
    L.check(L.la_state_pool_reorder(L.Slabs(dev), i32(slots), i32(parent), new, err))
    torch.cuda.synchronize()
    want, copies = R.reorder_ref(slots.tolist(), parent.tolist())
    assert int(err.item()) == 0 and new.tolist() == want
    for h, t in zip(host, dev):
        expect = h.clone()
        for s, d in copies:
            expect[d] = h[s]
        assert torch.equal(t.cpu(), expect)
        for b in range(B):
            for j in range(K):
                assert torch.equal(t[want[b][j]].cpu(), h[slots[b][parent[b][j]]])


def test_reorder_leaves_a_bad_sequence_alone():
    host = slabs_of(8, [64, 4096], 2)
    dev = [t.cuda() for t in host]
    new, err = i32(np.full((3, 2), 55)), i32([0])
    L.check(L.la_state_pool_reorder(L.Slabs(dev), i32([[0, 1], [2, 9], [4, 5]]), i32([[0, 0], [0, 0], [0, 2]]), new, err))
    torch.cuda.synchronize()
    assert int(err.item()) == L.DEVERR_READ_SLOT | L.DEVERR_TREE
    assert new.tolist() == [[0, 1], [-1, -1], [-1, -1]]
    for h, t in zip(host, dev):
        expect = h.clone()
        expect[1] = h[0]
        assert torch.equal(t.cpu(), expect)


@pytest.mark.parametrize("n_slots,n", [(1, 1), (5, 3), (40, 40), (1024, 7), (1025, 400), (5000, 2100), (3, 5), (0, 2)])
def test_alloc_share_free(n_slots, n):
    rng = np.random.RandomState(n_slots + n)
    ref = rng.randint(0, 3, n_slots) * (rng.rand(n_slots) < 0.5)
    free = [s for s in range(n_slots) if ref[s] == 0]
    r, slots, err = i32(ref), i32(np.full(n, 55)), i32([0])
    L.check(L.la_state_pool_alloc(r, slots, err))
    torch.cuda.synchronize()
    got = free[:n] + [-1] * max(0, n - len(free))
    assert slots.tolist() == got and int(err.item()) == (L.DEVERR_NO_SLOT if n > len(free) else 0)
    ref[free[:n]] = 1
    assert r.tolist() == ref.tolist()
    err.zero_()
    L.check(L.la_state_pool_share(r, slots, err))   # -1 is passed over
    L.check(L.la_state_pool_free(r, slots, err))
    L.check(L.la_state_pool_free(r, slots, err))
    torch.cuda.synchronize()
    ref[free[:n]] = 0
    assert int(err.item()) == 0 and r.tolist() == ref.tolist()


def test_counts_stay_sound():
    """The same slot often in one call, slots nobody holds, slots outside the pool."""
    r, err = i32([1, 0, 5, 2]), i32([0])
    L.check(L.la_state_pool_share(r, i32([2, 2, 0, 2, 3]), err))
    torch.cuda.synchronize()
    assert r.tolist() == [2, 0, 8, 3] and int(err.item()) == 0
    L.check(L.la_state_pool_share(r, i32([1] * 300), err))
    torch.cuda.synchronize()
    assert r.tolist() == [2, 0, 8, 3] and int(err.item()) == L.DEVERR_REF
    err.zero_()
    L.check(L.la_state_pool_free(r, i32([0, 0, 0, 0, 2]), err))
    torch.cuda.synchronize()
    assert r.tolist() == [0, 0, 7, 3] and int(err.item()) == L.DEVERR_REF
    err.zero_()
    L.check(L.la_state_pool_free(r, i32([4, -7, 3]), err))
    torch.cuda.synchronize()
    assert r.tolist() == [0, 0, 7, 2] and int(err.item()) == L.DEVERR_READ_SLOT


@pytest.mark.parametrize("spec", SPECS)
@pytest.mark.parametrize("n_slots,n", [(6, 1), (70, 20), (300, 90), (2500, 1100)])
def test_fork(n_slots, n, spec):
    if n_slots * sum(spec) > 1 << 26:
        spec = [64, 48]
    rng = np.random.RandomState(n_slots)
    held = rng.permutation(n_slots)[:n_slots // 2]
    ref = np.zeros(n_slots, int)
    ref[held] = rng.randint(1, 3, len(held))
    src = rng.choice(held, n)  # with repeats
    host = slabs_of(n_slots, spec, 3)
    dev = [t.cuda() for t in host]
    r, new, err = i32(ref), i32(np.full(n, 55)), i32([0])
    L.check(L.la_state_pool_fork(L.Slabs(dev), r, i32(src), new, err))
    torch.cuda.synchronize()
    free = [s for s in range(n_slots) if ref[s] == 0]
    got = (free + [-1] * n)[:n]
    assert new.tolist() == got and int(err.item()) == (0 if n <= len(free) else L.DEVERR_NO_SLOT)
    for h, t in zip(host, dev):
        expect = h.clone()
        for s, d in zip(src, got):
            if d >= 0:
                expect[d] = h[s]
        assert torch.equal(t.cpu(), expect)
    ref[free[:n]] = 1
    assert r.tolist() == ref.tolist()


def test_fork_of_slots_that_nothing_holds():
    """Such a source gets no slot, and could not be overwritten by another's copy."""
    host = slabs_of(6, [32, 64], 4)
    dev = [t.cuda() for t in host]
    r, new, err = i32([0, 1, 0, 2, 0, 0]), i32([55] * 5), i32([0])
    L.check(L.la_state_pool_fork(L.Slabs(dev), r, i32([3, 0, 1, 6, 1]), new, err))
    torch.cuda.synchronize()
    assert new.tolist() == [0, -1, 2, -1, 4] and int(err.item()) == L.DEVERR_REF | L.DEVERR_READ_SLOT
    assert r.tolist() == [1, 1, 1, 2, 1, 0]
    for h, t in zip(host, dev):
        assert torch.equal(t[0].cpu(), h[3]) and torch.equal(t[2].cpu(), h[1]) and torch.equal(t[4].cpu(), h[1])
        assert torch.equal(t[5].cpu(), h[5])


@pytest.mark.parametrize("spec", SPECS)
@pytest.mark.parametrize("n_slots,live", [(1, 0), (1, 1), (8, 3), (100, 50), (100, 100), (100, 0), (513, 200), (3000, 1700)])
def test_compact_and_remap(n_slots, live, spec):
    if n_slots * sum(spec) > 1 << 26:
        spec = [64, 48]
    rng = np.random.RandomState(n_slots + live)
    ref = np.zeros(n_slots, int)
    where = rng.permutation(n_slots)[:live]
    ref[where] = rng.randint(1, 4, live)
    host = slabs_of(n_slots, spec, 5)
    dev = [t.cuda() for t in host]
    new_ref, remap, moves = (i32(np.full(n_slots, 55)) for _ in range(3))
    counts, err = i32([55, 55]), i32([0])
    L.check(L.la_state_pool_compact(L.Slabs(dev), i32(ref), new_ref, remap, moves, counts, err))
    torch.cuda.synchronize()
    w_ref, w_remap, w_moves, w_counts = R.compact_ref(ref.tolist())
    assert int(err.item()) == 0 and counts.tolist() == w_counts
    assert new_ref.tolist() == w_ref and remap.tolist() == w_remap
    assert moves.tolist() == w_moves + [-1] * (n_slots - len(w_moves))
    for h, t in zip(host, dev):
        expect = h.clone()
        for s in w_moves:
            expect[w_remap[s]] = h[s]
        assert torch.equal(t.cpu(), expect)
    table = np.concatenate([where, [-1], where[:3]]).astype(int)
    t = i32(table)
    L.check(L.la_state_pool_remap(t, remap, t, err))  # in place
    torch.cuda.synchronize()
    assert t.tolist() == [w_remap[s] if s >= 0 else -1 for s in table] and int(err.item()) == 0
    out = i32([55] * 3)
    L.check(L.la_state_pool_remap(i32([n_slots, -5, -1]), remap, out, err))
    torch.cuda.synchronize()
    assert out.tolist() == [n_slots, -5, -1] and int(err.item()) == L.DEVERR_READ_SLOT


def test_many_slabs():
    host = slabs_of(12, [16 * (1 + i % 5) for i in range(L.MAX_SLABS)], 6)
    dev = [t.cuda() for t in host]
    ref = np.array([1, 0] * 6)
    outs = [i32(np.zeros(12)) for _ in range(3)]
    counts, err = i32([0, 0]), i32([0])
    L.check(L.la_state_pool_compact(L.Slabs(dev), i32(ref), *outs, counts, err))
    torch.cuda.synchronize()
    _, remap, moves, _ = R.compact_ref(ref.tolist())
    for h, t in zip(host, dev):
        expect = h.clone()
        for s in moves:
            expect[remap[s]] = h[s]
        assert torch.equal(t.cpu(), expect)


def test_beam_search_by_slots_is_beam_search_by_states():
    """Three steps of a toy decoder: select, reorder, decode step; captured once and replayed,
    against the same search that carries every beam's whole history of states along."""
    B, K, V, H, d = 2, 3, 97, 2, 64
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    emb = {n: unit(rnd(V, H, d)).cuda() for n in ("q", "k")}
    emb["v"] = rnd(V, H, d).cuda()
    head = (rnd(H * d, V) * 0.5).cuda()
    pool_t = (rnd(B * K, H, d, d) * 0.1).cuda()
    hist = torch.arange(B * K * 16, dtype=torch.float32).view(B * K, 16).cuda()
    pool = L.Pool(pool_t, H)
    slabs = L.Slabs([pool, hist])
    slots = [i32(np.arange(B * K).reshape(B, K)), i32(np.zeros((B, K)))]
    cum, fin = torch.tensor([[0.0] + [-float("inf")] * (K - 1)] * B).cuda(), i32(np.zeros((B, K)))
    x = rnd(B, K, V).cuda()
    parent, token, nfin = (i32(np.zeros((B, K))) for _ in range(3))
    score = torch.zeros(B, K, device="cuda")
    ws = torch.empty(L.la_beam_workspace_bytes(B, K, V, K), dtype=torch.uint8, device="cuda")
    err, o = i32([0]), torch.zeros(B * K, H, d, device="cuda")
    g, beta = torch.full((B * K, H), 0.9, device="cuda"), torch.full((B * K, H), 0.5, device="cuda")

    def step(src, dst):
        L.check(L.la_beam_select(x, cum, fin, 5, parent, token, score, nfin, ws))
        L.check(L.la_state_pool_reorder(slabs, src, parent, dst, err))
        cum.copy_(score)
        fin.copy_(nfin)
        t = token.view(-1).long()
        L.check(L.la_state_step("gated_delta", pool, dst.view(-1), pool, dst.view(-1), emb["q"][t], emb["k"][t],
                                emb["v"][t], g, beta, 1.0, o, err))
        x.copy_((o.view(B, K, H * d) @ head))

    states = pool_t.clone().cpu().double().view(B, K, H, d, d)
    hists = hist.clone().cpu().view(B, K, 16)
    for i in range(3):
        lx, lc, lf = x.cpu(), cum.cpu(), fin.cpu()
        step(slots[i % 2], slots[(i + 1) % 2])
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        par, tok, _, _, gap = R.beam_ref(lx, lc.numpy(), lf.numpy(), 5, K)
        assert gap > 1e-5
        np.testing.assert_array_equal(parent.cpu().numpy(), par)
        np.testing.assert_array_equal(token.cpu().numpy(), tok)
        now = torch.zeros_like(states)
        nh = torch.zeros_like(hists)
        for b in range(B):
            for j in range(K):
                S = states[b, par[b, j]] * 0.9
                t = tok[b, j]
                k, v = emb["k"][t].cpu().double(), emb["v"][t].cpu().double()
                u = 0.5 * (v - (S * k[:, :, None]).sum(1))
                now[b, j] = S + k[:, :, None] * u[:, None, :]
                nh[b, j] = hists[b, par[b, j]]
        states, hists = now, nh
        at = slots[(i + 1) % 2].cpu().long()
        assert torch.equal(hist.cpu()[at], hists)
        torch.testing.assert_close(pool_t.cpu().double()[at], states, rtol=0, atol=1e-4)


def test_fork_step_free_compact_on_a_captured_stream():
    """A branch is tried and released, requests leave, the pool is compacted: captured together
    and replayed on other counts."""
    n_slots, H, d = 40, 2, 64
    gen = torch.Generator().manual_seed(9)
    base = torch.randn(n_slots, H, d, d, generator=gen)
    pool_t = base.cuda()
    pool = L.Pool(pool_t, H)
    slabs = L.Slabs([pool])
    ref, src, new = i32(np.zeros(n_slots)), i32([0] * 4), i32([0] * 4)
    new_ref, remap, moves = (i32(np.zeros(n_slots)) for _ in range(3))
    counts, err, gone = i32([0, 0]), i32([0]), i32([0] * 5)
    table, new_table = i32([0] * 10), i32([0] * 10)

    def body():
        L.check(L.la_state_pool_fork(slabs, ref, src, new, err))
        L.check(L.la_state_pool_free(ref, gone, err))
        L.check(L.la_state_pool_compact(slabs, ref, new_ref, remap, moves, counts, err))
        L.check(L.la_state_pool_remap(table, remap, new_table, err))

    rng = np.random.RandomState(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        ref.fill_(0)
        ref[:10] = 1
        gone.copy_(torch.arange(5))
        src.copy_(torch.arange(4) + 5)
        body()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            body()
    for _ in range(3):
        held = rng.permutation(n_slots)[:15]
        counts0 = np.zeros(n_slots, int)
        counts0[held] = 1
        sources, leaving = rng.choice(held, 4), held[:5]
        keep = held[5:]
        pool_t.copy_(base)
        ref.copy_(torch.tensor(counts0))
        src.copy_(torch.tensor(sources))
        gone.copy_(torch.tensor(leaving))
        table.copy_(torch.tensor(keep))
        err.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        free = [s for s in range(n_slots) if counts0[s] == 0]
        assert new.tolist() == free[:4]
        content = {s: base[s] for s in keep}
        for s, dd in zip(sources, free[:4]):
            content[dd] = base[s]
            counts0[dd] = 1
        counts0[leaving] = 0
        w_ref, w_remap, _, w_counts = R.compact_ref(counts0.tolist())
        assert counts.tolist() == w_counts and new_ref.tolist() == w_ref
        assert new_table.tolist() == [w_remap[s] for s in keep]
        for s, x in content.items():
            assert torch.equal(pool_t[w_remap[s]].cpu(), x)
