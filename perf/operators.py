"""Serving operators around the recurrent-state slot pool, as measured cases.

Five calls of a serving loop of linear-attention layers:
  tree     la_state_tree: a packed batch of drafted token trees read against the slot pool
           (speculative decoding's verification), outputs of every node and its write vector u
  commit   la_tree_accept + la_state_tree_commit: the drafted path the target agrees with,
           and the state at its end, from the kept write vectors
  beam     la_beam_select + la_state_pool_reorder: the best continuations over beams and
           vocabulary, and the layers' states moved to the beams that go on
  fork     la_state_pool_fork + la_state_pool_free: new slots holding copies of live ones over
           all layers, released again (a branch that was tried)
  compact  la_state_pool_compact + la_state_pool_remap: live slots moved to the front of the
           pools, the request table following

With `own` false every call is computed in its plain form, elementary torch operations in 32
bits (the beam scores in 64: values next to a border decide whole numbers).
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _size(t):
    return torch.finfo(DT[t]).bits // 8


# ---- cases ---------------------------------------------------------------------------

def listed():
    return [
        # one interactive request, a small draft: latency
        dict(name="tree 1x8", op="tree", B=1, lo=8, hi=8, Hqk=16, Hv=32, dk=128, dv=128, state="bf16", io="bf16",
             rule="gated_delta", shape="tree"),
        # the decode64 batch with ragged drafts of up to 32 tokens
        dict(name="tree 64 ragged", op="tree", B=64, lo=1, hi=32, Hqk=16, Hv=32, dk=128, dv=128, state="bf16",
             io="bf16", rule="gated_delta", shape="tree"),
        # a full server, the largest drafts
        dict(name="tree 256x64", op="tree", B=256, lo=33, hi=64, Hqk=16, Hv=32, dk=128, dv=128, state="bf16",
             io="bf16", rule="gated_delta", shape="tree"),
        # the channel-wise gate in FP32 throughout
        dict(name="tree kda f32", op="tree", B=16, lo=1, hi=24, Hqk=8, Hv=8, dk=128, dv=128, state="f32", io="f32",
             rule="kda", shape="tree"),
        # acceptance and the new states of the decode64 batch
        dict(name="commit 64", op="commit", B=64, lo=1, hi=32, Hqk=16, Hv=32, dk=128, dv=128, state="bf16", io="bf16",
             rule="gated_delta", shape="tree"),
        # the mamba2 layer's heads (gated rule, 128 x 64) in FP32
        dict(name="commit mamba2 f32", op="commit", B=32, lo=4, hi=16, Hqk=1, Hv=128, dk=128, dv=64, state="f32",
             io="f32", rule="gated", shape="chain"),
        # one request, four beams, one layer: latency
        dict(name="beam 1x4", op="beam", B=1, K=4, V=32000, io="f32", layers=1, Hv=32, d=128),
        # a batch with eight beams each, an odd vocabulary, two layers
        dict(name="beam 48x8", op="beam", B=48, K=8, V=50257, io="bf16", layers=2, Hv=32, d=128),
        # one branch of one request, one small layer: latency
        dict(name="fork 1", op="fork", n=1, slots=64, layers=1, Hv=4, d=64, state="bf16"),
        # 64 branches over eight layers, states and convolution histories
        dict(name="fork 64x8", op="fork", n=64, slots=160, layers=8, Hv=32, d=128, state="bf16"),
        # a small pool shrunk: latency
        dict(name="compact 64", op="compact", slots=64, live=20, layers=1, Hv=4, d=64, state="bf16"),
        # half of a 512-slot pool left by finished requests, two layers
        dict(name="compact 512x2", op="compact", slots=512, live=256, layers=2, Hv=32, d=128, state="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "commit", "beam", "fork", "compact"])
    if op in ("tree", "commit"):
        rule = rng.choice(["gated_delta", "gated_delta", "gated", "delta", "linear", "kda"])
        dk, dv = rng.choice([(128, 128), (128, 128), (128, 64), (64, 64)])
        hi = _log_int(rng, 1, 64)
        lo = rng.choice([hi, max(1, hi // 2), 1])
        Hqk = rng.choice([1, 2, 4, 8, 16])
        Hv = Hqk * rng.choice([1, 2, 4])
        state = rng.choice(["bf16", "bf16", "f32"])
        io = rng.choice(["bf16", "bf16", "f32"])
        B = _log_int(rng, 1, 256)
        if rule == "kda":  # the plain form holds n x n decays for each channel
            while B * Hv * dk * hi * hi > 1 << 27:
                B, hi, lo = max(1, B // 2), max(1, hi - hi // 4), 1
        case = dict(op=op, B=B, lo=lo, hi=hi, Hqk=Hqk, Hv=Hv, dk=dk, dv=dv, state=state, io=io, rule=rule,
                    shape=rng.choice(["tree", "tree", "chain"]))
        while work(case)["bytes"] > 7e8:
            case["B"] -= case["B"] // 4
        return case
    if op == "beam":
        K = rng.randint(2, 16)
        B = _log_int(rng, 1, 64)
        V = _log_int(rng, 1000, 160000)
        while B * K > 384 or B * K * V > 24_000_000:
            B, V = max(1, B - max(1, B // 3)), max(1000, V - V // 8)
        return dict(op=op, B=B, K=K, V=V, io=rng.choice(["bf16", "f32"]), layers=rng.randint(1, 2),
                    Hv=rng.choice([4, 8, 16, 32]), d=rng.choice([64, 128]))
    slots = _log_int(rng, 16, 512)
    layers = rng.randint(1, 8)
    Hv = rng.choice([2, 4, 8, 16, 32])
    d = rng.choice([64, 128])
    state = rng.choice(["bf16", "f32"])
    while slots * layers * Hv * d * d * _size(state) > 1 << 30:
        slots, layers = max(16, slots - slots // 4), max(1, layers - 1)
    if op == "fork":
        return dict(op=op, n=rng.randint(1, max(1, slots // 3)), slots=slots, layers=layers, Hv=Hv, d=d, state=state)
    return dict(op=op, slots=slots, live=rng.randint(1, slots - 1), layers=layers, Hv=Hv, d=d, state=state)


# ---- inputs --------------------------------------------------------------------------

def _lens(case):
    lo, hi, B = case["lo"], case["hi"], case["B"]
    return [hi if b == 0 else lo + (b * 7919) % (hi - lo + 1) for b in range(B)]


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-30)


def _tree_state(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 32))
    B, Hqk, Hv, dk, dv = (case[n] for n in ("B", "Hqk", "Hv", "dk", "dv"))
    lens = _lens(case)
    T = sum(lens)
    st, io = DT[case["state"]], DT[case["io"]]
    slots = 2 * B + 3
    pool = (_randn(gen, slots, Hv, dk, dv) * 0.05).to(st)
    perm = rs.permutation(slots)
    # a drafter's tree: every node continues a random earlier one (or the request's last
    # token, -1); a chain is a drafter without branches
    parent = [(i - 1 if case["shape"] == "chain" else int(rs.randint(-1, i)) if i else -1) for n in lens for i in range(n)]
    # drafted tokens differ among all nodes of a tree; the target agrees with one child of
    # most nodes
    draft, target, root = [], [], []
    at = 0
    for n in lens:
        tok = rs.choice(32000, size=n + 1, replace=False)
        kids = {p: [i for i in range(n) if parent[at + i] == p] for p in range(-1, n)}
        want = {p: int(tok[rs.choice(c)]) if c and rs.rand() < 0.75 else int(tok[n]) for p, c in kids.items()}
        draft += [int(t) for t in tok[:n]]
        target += [want[i] for i in range(n)]
        root.append(want[-1])
        at += n
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    gshape = (T, Hv, dk) if case["rule"] == "kda" else (T, Hv)
    s = dict(case=case, T=T, n=max(lens), pool=pool, read=dev(perm[:B].copy()), cu=dev(np.concatenate([[0], np.cumsum(lens)])),
             parent=dev(parent),
             k=_unit(_randn(gen, T, Hqk, dk)).to(io), g=torch.exp(-torch.nn.functional.softplus(_randn(gen, *gshape))),
             beta=torch.sigmoid(_randn(gen, T, Hv)), scale=1.0)
    if case["op"] == "tree":
        s |= dict(q=_unit(_randn(gen, T, Hqk, dk)).to(io), v=_randn(gen, T, Hv, dv).to(io),
                  o=torch.zeros(T, Hv, dv, dtype=io, device="cuda"), u=torch.zeros(T, Hv, dv, device="cuda"))
    else:
        s |= dict(u=_randn(gen, T, Hv, dv) * 0.5, draft=dev(draft), target=dev(target), root=dev(root),
                  dst=torch.zeros(B, Hv, dk, dv, dtype=st, device="cuda"),
                  leaf=torch.zeros(B, dtype=torch.int32, device="cuda"), count=torch.zeros(B, dtype=torch.int32, device="cuda"),
                  next=torch.zeros(B, dtype=torch.int32, device="cuda"))
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def _layer_slabs(gen, case, slots):
    """Every layer's state pool and the history of its short convolution (width 4)."""
    H, d = case["Hv"], case["d"]
    st = DT[case.get("state", "bf16")]
    slabs = []
    for _ in range(case["layers"]):
        slabs.append(torch.empty(slots, H, d, d, dtype=st, device="cuda").normal_(0, 0.05, generator=gen))
        slabs.append(torch.empty(slots, H, 3 * d, 3, dtype=torch.bfloat16, device="cuda").normal_(generator=gen))
    return slabs


def prepare(case, seed):
    if case["op"] in ("tree", "commit"):
        return _tree_state(case, seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 32))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ints = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] == "beam":
        B, K, V = case["B"], case["K"], case["V"]
        logits = _randn(gen, B, K, V) * 2.5
        # a constrained decoder masks a part of the vocabulary
        logits[torch.rand(B, K, V, generator=gen, device="cuda") < 0.02] = float("-inf")
        cum = -_randn(gen, B, K).abs().cumsum(1) * 0.5 - 3.0
        cum[7::8, 1:] = float("-inf")  # requests in their first step: one live beam
        cum[7::8, 0] = 0.0
        finished = (torch.rand(B, K, generator=gen, device="cuda") < 0.1).to(torch.int32)
        finished[7::8] = 0
        slots = B * K + 5
        z32 = lambda *sh: torch.zeros(*sh, dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(case=case, logits=logits.to(DT[case["io"]]), cum=cum, finished=finished, eos=2,
                    slots=ints(rs.permutation(slots)[:B * K].reshape(B, K)), slabs=_layer_slabs(gen, case, slots), err=err,
                    parent=z32(B, K), token=z32(B, K), score=torch.zeros(B, K, device="cuda"), finished_out=z32(B, K),
                    new_slots=z32(B, K))
    slots = case["slots"]
    live = case["live"] if case["op"] == "compact" else min(slots - case["n"], max(1, slots // 2))
    ref = np.zeros(slots, np.int32)
    where = rs.permutation(slots)[:live]
    ref[where] = rs.randint(1, 4, live)
    s = dict(case=case, ref=ints(ref), slabs=_layer_slabs(gen, case, slots), err=err)
    if case["op"] == "fork":
        s |= dict(src=ints(rs.choice(where, case["n"])), new=ints(np.zeros(case["n"])))
    else:
        table = np.concatenate([where, rs.choice(where, live // 2 + 1), [-1]])
        s |= dict(table=ints(table), new_table=ints(np.zeros(len(table))), new_ref=ints(np.zeros(slots)),
                  remap=ints(np.zeros(slots)), moves=ints(np.zeros(slots)), counts=ints(np.zeros(2)))
    return s


# ---- the framework's calls ---------------------------------------------------------------

def _handles(s):
    """What a program makes once of its buffers: pools, slab lists and workspaces."""
    from gated_deltanet_recurrent_la_b200 import lastate as L
    c = s["case"]
    h = {}
    if c["op"] in ("tree", "commit"):
        h["src"] = L.Pool(s["pool"], c["Hqk"])
        if c["op"] == "commit":
            h["dst"] = L.Pool(s["dst"], c["Hqk"])
    else:
        h["slabs"] = L.Slabs(s["slabs"])
        if c["op"] == "beam":
            n = L.la_beam_workspace_bytes(c["B"], c["K"], c["V"], c["K"])
            h["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    s["handles"] = h
    return h


def _run_own(s):
    from gated_deltanet_recurrent_la_b200 import lastate as L
    c, h = s["case"], s.get("handles") or _handles(s)
    if c["op"] == "tree":
        L.check(L.la_state_tree(c["rule"], h["src"], s["read"], s["cu"], s["parent"], s["n"], s["q"], s["k"], s["v"],
                                s["g"], s["beta"], s["scale"], s["o"], s["u"], s["err"]))
        return {"o": s["o"], "u": s["u"]}
    if c["op"] == "commit":
        L.check(L.la_tree_accept(s["cu"], s["parent"], s["n"], s["draft"], s["target"], s["root"], s["leaf"], s["count"],
                                 s["next"], s["err"]))
        L.check(L.la_state_tree_commit(c["rule"], h["src"], s["read"], h["dst"], None, s["cu"], s["parent"], s["leaf"],
                                       s["n"], s["k"], s["g"], s["u"], s["err"]))
        return {"leaf": s["leaf"], "count": s["count"], "next": s["next"], "state": s["dst"]}
    if c["op"] == "beam":
        L.check(L.la_beam_select(s["logits"], s["cum"], s["finished"], s["eos"], s["parent"], s["token"], s["score"],
                                 s["finished_out"], h["ws"]))
        L.check(L.la_state_pool_reorder(h["slabs"], s["slots"], s["parent"], s["new_slots"], s["err"]))
        return {"parent": s["parent"], "token": s["token"], "score": s["score"], "finished": s["finished_out"],
                "slots": s["new_slots"], "slabs": s["slabs"]}
    if c["op"] == "fork":
        L.check(L.la_state_pool_fork(h["slabs"], s["ref"], s["src"], s["new"], s["err"]))
        L.check(L.la_state_pool_free(s["ref"], s["new"], s["err"]))
        return {"new": s["new"], "ref": s["ref"], "slabs": s["slabs"]}
    L.check(L.la_state_pool_compact(h["slabs"], s["ref"], s["new_ref"], s["remap"], s["moves"], s["counts"], s["err"]))
    L.check(L.la_state_pool_remap(s["table"], s["remap"], s["new_table"], s["err"]))
    return {"ref": s["new_ref"], "remap": s["remap"], "moves": s["moves"], "counts": s["counts"],
            "table": s["new_table"], "slabs": s["slabs"]}


# ---- the plain forms -----------------------------------------------------------------------

def _closure(N, x, bits):
    """(I - N)^-1 x for a strictly lower N of a tree (nilpotent): (I + N)(I + N^2)(I + N^4)..."""
    for _ in range(bits):
        x = x + N @ x
        N = N @ N
    return x


def _padded(s):
    """Index of node i of request b in the packed arrays [B, n], whether there is one, the
    request and place of every packed row, and P[b, t, s] = 1 where s is t's parent."""
    n, T = s["n"], s["T"]
    cu = s["cu"].long()
    i = torch.arange(n, device="cuda")
    there = i < (cu[1:] - cu[:-1])[:, None]
    at = (cu[:-1, None] + i).clamp(max=T - 1)
    rows = torch.arange(T, device="cuda")
    req = torch.searchsorted(cu[1:].contiguous(), rows, right=True)
    parent = torch.where(there, s["parent"][at].long(), -2)
    P = (parent[:, :, None] == i).float()
    return at, there, req, rows - cu[req], parent, P


def _plain_decays(s, at, there, parent, P, bits):
    """D[b, h, (channel,) t, s], the product of the gates on the path from s (exclusive) to t
    (0 off the path, 1 on the diagonal), and Gamma[b, h, (channel,) t], from the root."""
    rule, B, Hv = s["case"]["rule"], s["case"]["B"], s["case"]["Hv"]
    n = P.shape[1]
    if rule == "kda":
        g = s["g"][at].permute(0, 2, 3, 1)                      # [B, H, dk, n]
        PP = P[:, None, None]
        root = (parent == -1).float()[:, None, None]
    else:
        g = s["g"][at].permute(0, 2, 1) if rule in ("gated", "gated_delta") else torch.ones(B, Hv, n, device="cuda")
        PP = P[:, None]
        root = (parent == -1).float()[:, None]
    D = _closure(PP * g[..., None], torch.eye(n, device="cuda").expand(*g.shape, n), bits)
    return D, (D @ (g * root)[..., None])[..., 0]


def _plain_tree(s):
    c = s["case"]
    rule, B, Hqk, Hv = c["rule"], c["B"], c["Hqk"], c["Hv"]
    at, there, req, pos, parent, P = _padded(s)
    bits = max(1, (s["n"] - 1).bit_length())
    heads = lambda x: x[at].float().permute(0, 2, 1, 3)  # noqa: E731
    q, k = (heads(s[x]).repeat_interleave(Hv // Hqk, 1) for x in ("q", "k"))
    v = heads(s["v"]) * there[:, None, :, None]
    S0 = s["pool"][s["read"].long()].float()
    D, G = _plain_decays(s, at, there, parent, P, bits)
    strict = 1 - torch.eye(s["n"], device="cuda")
    if rule == "kda":
        kD = D.permute(0, 1, 3, 4, 2) * k[:, :, None]           # [B, H, t, s, dk]
        KK = (kD * k[:, :, :, None]).sum(-1)
        QK = (kD * q[:, :, :, None]).sum(-1)
        Gt = G.transpose(2, 3)
        KS, QS = (k * Gt) @ S0, (q * Gt) @ S0
    else:
        KK, QK = D * (k @ k.transpose(2, 3)), D * (q @ k.transpose(2, 3))
        KS, QS = G[..., None] * (k @ S0), G[..., None] * (q @ S0)
    if rule in ("linear", "gated"):
        U = v
    else:
        b = (s["beta"][at] * there[..., None]).permute(0, 2, 1)[..., None]
        U = _closure(-b * KK * strict, b * (v - KS), bits)
    o = s["scale"] * (QS + QK @ U)
    return {"o": o[req, :, pos].to(DT[c["io"]]), "u": U[req, :, pos].contiguous()}


def _plain_commit(s):
    c = s["case"]
    Hqk, Hv = c["Hqk"], c["Hv"]
    at, there, req, pos, parent, P = _padded(s)
    n = s["n"]
    bits = max(1, (n - 1).bit_length())
    draft, target = s["draft"][at], s["target"][at]
    # a node is agreed to if its token is what the target wants after its parent and no
    # earlier child of that parent has the same token; it is accepted if its whole path is
    want = torch.where(parent >= 0, target.gather(1, parent.clamp(min=0)), s["root"][:, None])
    i = torch.arange(n, device="cuda")
    twin = (parent[:, :, None] == parent[:, None, :]) & (draft[:, :, None] == draft[:, None, :]) & (i[None, :] < i[:, None])
    ok = there & (draft == want) & ~twin.any(2)
    anc = _closure(P, torch.eye(n, device="cuda").expand(P.shape), bits)     # ancestor or self
    taken = (anc @ (~ok).float()[..., None])[..., 0] == 0
    leaf = torch.where(taken & there, i, -1).amax(1)
    on = anc.gather(1, leaf.clamp(min=0)[:, None, None].expand(-1, 1, n))[:, 0] * (leaf >= 0)[:, None]
    count = on.sum(1)
    nxt = torch.where(leaf >= 0, target.gather(1, leaf.clamp(min=0)[:, None])[:, 0], s["root"])
    D, G = _plain_decays(s, at, there, parent, P, bits)
    S0 = s["pool"][s["read"].long()].float()
    k = s["k"][at].float().permute(0, 2, 1, 3).repeat_interleave(Hv // Hqk, 1)
    u = s["u"][at].permute(0, 2, 1, 3)
    b = torch.arange(c["B"], device="cuda")
    row = leaf.clamp(min=0)
    if c["rule"] == "kda":
        k = k * (D[b, :, :, row] * on[:, None, None]).transpose(2, 3)
        G = G[b, :, :, row][..., None]
    else:
        k = k * (D[b, :, row] * on[:, None])[..., None]
        G = G[b, :, row][..., None, None]
    G = torch.where((leaf >= 0)[:, None, None, None], G, 1.0)
    state = G * S0 + k.transpose(2, 3) @ u
    return {"leaf": leaf.int(), "count": count.int(), "next": nxt.int(), "state": state.to(DT[c["state"]])}


def _plain_beam(s):
    c = s["case"]
    B, K, V = c["B"], c["K"], c["V"]
    minus = float("-inf")
    x = torch.where((s["cum"] == minus)[..., None], minus, s["logits"].float())
    top = x.amax(2, keepdim=True).double()
    lse = torch.where(top == minus, 0.0, top + (x.double() - top.clamp(min=-3e38)).exp().sum(2, keepdim=True).log())
    done = s["finished"][..., None] != 0
    eos = (torch.arange(V, device="cuda") == s["eos"]).expand(B, K, V)
    x = torch.where(done, torch.where(eos & (s["cum"] != minus)[..., None], 0.0, minus), x)
    lse = torch.where(done, 0.0, lse)
    # the best K of each beam: a key that orders values, then the lower index
    bits = x.view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    order = torch.where(x == 0, 0, order)
    key = (order << 32) | (0xFFFFFFFF - torch.arange(V, device="cuda"))
    idx = key.topk(K, dim=2, sorted=True)[1]
    score = s["cum"].double()[..., None] + x.gather(2, idx).double() - lse
    rank = torch.sort(score.reshape(B, K * K), dim=1, descending=True, stable=True)
    pick = rank[1][:, :K]
    parent = pick // K
    token = idx.reshape(B, K * K).gather(1, pick)
    fin = (s["finished"].gather(1, parent) != 0) | (token == s["eos"])
    # the first child of a beam stays in its slot; the others take the slots of the beams
    # without children, both in increasing order
    j = torch.arange(K, device="cuda")
    same = parent[:, :, None] == parent[:, None, :]
    first = ~(same & (j[None, :] < j[:, None])).any(2)
    dead = ~(parent[:, None, :] == j[:, None]).any(2)
    dead_list = torch.sort((~dead).int(), dim=1, stable=True)[1]
    nth = ((~first).long().cumsum(1) - 1).clamp(min=0)
    old = s["slots"].long()
    frm = old.gather(1, parent)
    new = torch.where(first, frm, old.gather(1, dead_list.gather(1, nth)))
    for t in s["slabs"]:
        t[new.reshape(-1)] = t[frm.reshape(-1)]
    return {"parent": parent.int(), "token": token.int(), "score": rank[0][:, :K].float(), "finished": fin.int(),
            "slots": new.int(), "slabs": s["slabs"]}


def _plain_fork(s):
    n = s["case"]["n"]
    new = torch.sort((s["ref"] != 0).int(), stable=True)[1][:n]
    s["ref"][new] = 1
    src = s["src"].long()
    for t in s["slabs"]:
        t[new] = t[src]
    s["ref"].index_add_(0, new, torch.full((n,), -1, dtype=torch.int32, device="cuda"))
    return {"new": new.int(), "ref": s["ref"], "slabs": s["slabs"]}


def _plain_compact(s):
    ref = s["ref"]
    n = ref.numel()
    at = torch.arange(n, device="cuda")
    live = ref > 0
    n_live = live.sum()
    hole, tail = ~live & (at < n_live), live & (at >= n_live)
    holes = torch.sort((~hole).int(), stable=True)[1]
    remap = torch.where(tail, holes[(tail.long().cumsum(0) - 1).clamp(min=0)], torch.where(live, at, -1))
    moved = tail.sum()
    moves = torch.where(at < moved, torch.sort((~tail).int(), stable=True)[1], -1)
    new_ref = torch.zeros_like(ref)
    new_ref[remap[live]] = ref[live]
    src = tail.nonzero()[:, 0]
    for t in s["slabs"]:
        t[remap[src]] = t[src]
    table = s["table"].long()
    table = torch.where(table >= 0, remap[table.clamp(min=0)], table)
    return {"ref": new_ref, "remap": remap.int(), "moves": moves.int(), "counts": torch.stack([n_live, moved]).int(),
            "table": table.int(), "slabs": s["slabs"]}


PLAIN = {"tree": _plain_tree, "commit": _plain_commit, "beam": _plain_beam, "fork": _plain_fork, "compact": _plain_compact}


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("tree", "commit"):
        lens, Hqk, Hv, dk, dv = _lens(case), case["Hqk"], case["Hv"], case["dk"], case["dv"]
        sb, ib, T, B = _size(case["state"]), _size(case["io"]), sum(lens), case["B"]
        gates = {"linear": 0, "gated": 1, "delta": 0, "gated_delta": 1, "kda": dk}[case["rule"]]
        betas = 1 if "delta" in case["rule"] or case["rule"] == "kda" else 0
        state = B * Hv * dk * dv
        if op == "tree":
            # the state once, q and k once per q/k head, v, o, u; three products with the
            # state or among the nodes (a node meets its path, about 3 + ln n nodes of a tree)
            path = sum(n * (n / 2 if case["shape"] == "chain" else 3 + math.log(n)) for n in lens)
            return {"bytes": state * sb + T * (2 * Hqk * dk * ib + 2 * Hv * dv * ib + Hv * dv * 4 + 4 * Hv * (gates + betas) + 4),
                    "flops": 4 * T * Hv * dk * dv + path * Hv * (4 * dk + 4 * dv)}
        taken = 2 * B  # nodes accepted, about
        return {"bytes": 2 * state * sb + taken * (Hqk * dk * ib + Hv * dv * 4 + 4 * Hv * gates) + 12 * T,
                "flops": state + 2 * taken * Hv * dk * dv}
    slab = lambda st: case["layers"] * (case["Hv"] * case["d"] ** 2 * st + case["Hv"] * 3 * case["d"] * 3 * 2)  # noqa: E731
    if op == "beam":
        # about 0.4 of the beams die and are overwritten
        return {"bytes": case["B"] * case["K"] * (case["V"] * _size(case["io"]) + 24) + 0.4 * case["B"] * case["K"] * 2 * slab(2),
                "flops": 4 * case["B"] * case["K"] * case["V"]}
    if op == "fork":
        return {"bytes": case["n"] * (2 * slab(_size(case["state"])) + 12), "flops": 0}
    moved = case["live"] * (1 - case["live"] / case["slots"])
    return {"bytes": max(1.0, moved) * 2 * slab(_size(case["state"])) + 16 * case["slots"], "flops": 0}


# ---- the definition in 64 bits -----------------------------------------------------------------

def _exact_tree(s):
    """Node by node on explicit states: S <- Diag(a) S_parent + k u^T, one request at a time."""
    c = s["case"]
    rule, ratio = c["rule"], c["Hv"] // c["Hqk"]
    cu, parent = s["cu"].tolist(), s["parent"].tolist()
    q, k = (s[x].double().repeat_interleave(ratio, 1) for x in ("q", "k"))
    v, g, beta = s["v"].double(), s["g"].double(), s["beta"].double()
    o, u = torch.zeros_like(v), torch.zeros_like(v)
    for b, slot in enumerate(s["read"].tolist()):
        states = {-1: s["pool"][slot].double()}
        for t in range(cu[b], cu[b + 1]):
            S = states[parent[t]]
            if rule == "kda":
                S = S * g[t][:, :, None]
            elif rule in ("gated", "gated_delta"):
                S = S * g[t][:, None, None]
            w = v[t]
            if rule in ("delta", "gated_delta", "kda"):
                w = beta[t][:, None] * (w - (S * k[t][:, :, None]).sum(1))
            S = S + k[t][:, :, None] * w[:, None, :]
            states[t - cu[b]] = S
            u[t], o[t] = w, s["scale"] * (S * q[t][:, :, None]).sum(1)
    return {"o": o, "u": u}


def _exact_commit(s):
    c = s["case"]
    rule, ratio = c["rule"], c["Hv"] // c["Hqk"]
    cu, parent, draft, target, root = (s[x].tolist() for x in ("cu", "parent", "draft", "target", "root"))
    k, u, g = s["k"].double().repeat_interleave(ratio, 1), s["u"].double(), s["g"].double()
    out = torch.zeros(s["dst"].shape, dtype=torch.float64, device="cuda")
    for b, slot in enumerate(s["read"].tolist()):
        S, at, want = s["pool"][slot].double(), -1, root[b]
        while True:
            nxt = [t for t in range(cu[b], cu[b + 1]) if parent[t] == at and draft[t] == want]
            if not nxt:
                break
            t = nxt[0]
            if rule == "kda":
                S = S * g[t][:, :, None]
            elif rule in ("gated", "gated_delta"):
                S = S * g[t][:, None, None]
            S = S + k[t][:, :, None] * u[t][:, None, :]
            at, want = t - cu[b], target[t]
        out[b] = S
    return {"leaf": None, "count": None, "next": None, "state": out}


def _exact_beam(s):
    B, K, V = s["logits"].shape
    best = []
    for b in range(B):
        x = s["logits"][b].double()
        x[s["cum"][b] == float("-inf")] = float("-inf")
        lp = torch.log_softmax(x, 1).nan_to_num(nan=float("-inf"), neginf=float("-inf"))
        done = s["finished"][b] != 0
        lp[done] = float("-inf")
        lp[done, s["eos"]] = 0.0
        total = (lp + s["cum"][b].double()[:, None]).reshape(-1)
        best.append(total.topk(K).values)
    return {"parent": None, "token": None, "score": torch.stack(best), "finished": None, "slots": None, "slabs": None}


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None
    s = prepare(case, seed)
    if case["op"] == "beam":
        return _exact_beam(s)
    return _exact_tree(s) if case["op"] == "tree" else _exact_commit(s)
