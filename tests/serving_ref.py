"""Plain implementations in 64 bits of the serving operators (drafted trees, beam selection,
slot bookkeeping), written from their definitions, and the inputs of their tests."""
import numpy as np
import torch

RULES = ("linear", "gated", "delta", "gated_delta", "kda")


def uses_gate(rule):
    return rule in ("gated", "gated_delta", "kda")


def uses_beta(rule):
    return rule in ("delta", "gated_delta", "kda")


def random_parents(rng, n, shape):
    if shape == "chain":
        return [i - 1 for i in range(n)]
    if shape == "star":
        return [-1] * n
    return [int(rng.randint(-1, i)) if i else -1 for i in range(n)]


def tree_inputs(*, lens, Hqk, Hv, dk, dv, rule, state_dtype, io_dtype, seed, shape="tree", wide=False, slots=None):
    """Host tensors of a packed batch of trees.  wide: gates in [-1, 1] with zeros, beta in [0, 2]."""
    rng = np.random.RandomState(seed)
    gen = torch.Generator().manual_seed(seed)
    T, B = sum(lens), len(lens)
    slots = 2 * B + 1 if slots is None else slots
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-30)  # noqa: E731
    gshape = (T, Hv, dk) if rule == "kda" else (T, Hv)
    if wide:
        g = torch.rand(*gshape, generator=gen) * 2 - 1
        g = torch.where(torch.rand(*gshape, generator=gen) < 0.1, torch.zeros(()), g)
        beta = torch.rand(T, Hv, generator=gen) * 2
    else:
        g = torch.exp(-torch.nn.functional.softplus(r(*gshape)))
        beta = torch.sigmoid(r(T, Hv))
    return dict(rule=rule, Hqk=Hqk, Hv=Hv, dk=dk, dv=dv, T=T, B=B, n=max(lens + [1]), scale=0.75,
                cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32),
                parent=torch.tensor([p for n in lens for p in random_parents(rng, n, shape)], dtype=torch.int32),
                pool=(r(slots, Hv, dk, dv) * 0.3).to(state_dtype),
                read=torch.tensor(rng.permutation(slots)[:B].copy(), dtype=torch.int32),
                q=unit(r(T, Hqk, dk)).to(io_dtype), k=unit(r(T, Hqk, dk)).to(io_dtype), v=r(T, Hv, dv).to(io_dtype),
                g=g.contiguous(), beta=beta.contiguous())


def decayed(rule, S, g):
    if rule == "kda":
        return S * g[:, :, None]
    return S * g[:, None, None] if uses_gate(rule) else S


def tree_ref(inp, states):
    """Node by node on explicit FP64 states (states [slots, Hv, dk, dv]): o, u, and the bounds
    mag_o, mag_u of their rounding errors (the same recurrences on absolute values), and the
    depth of the deepest node."""
    ratio = inp["Hv"] // inp["Hqk"]
    q, k = (inp[x].double().repeat_interleave(ratio, 1) for x in ("q", "k"))
    v, g, beta = inp["v"].double(), inp["g"].double(), inp["beta"].double()
    cu, parent = inp["cu"].tolist(), inp["parent"].tolist()
    o, u, mo, mu = (torch.zeros_like(v) for _ in range(4))
    depth = 0
    for b in range(inp["B"]):
        S0 = states[int(inp["read"][b])].double()
        S, M, D = {-1: S0}, {-1: S0.abs()}, {-1: 0}
        for t in range(cu[b], cu[b + 1]):
            p = parent[t]
            s, m = decayed(inp["rule"], S[p], g[t]), decayed(inp["rule"], M[p], g[t].abs())
            w, mw = v[t], v[t].abs()
            if uses_beta(inp["rule"]):
                w = beta[t][:, None] * (w - (s * k[t][:, :, None]).sum(1))
                mw = beta[t][:, None] * (mw + (m * k[t].abs()[:, :, None]).sum(1))
            i = t - cu[b]
            S[i] = s + k[t][:, :, None] * w[:, None, :]
            M[i] = m + k[t].abs()[:, :, None] * mw[:, None, :]
            D[i] = D[p] + 1
            depth = max(depth, D[i])
            u[t], mu[t] = w, mw
            o[t] = inp["scale"] * (S[i] * q[t][:, :, None]).sum(1)
            mo[t] = inp["scale"] * (M[i] * q[t].abs()[:, :, None]).sum(1)
    return o, u, mo, mu, depth


def tree_steps(depth, dk):
    """FP32 roundings that reach a node's outputs, as multiples of 2^-24 of its magnitude bound:
    a node's own sums have at most dk + depth terms of up to depth decay products each, and
    every node above adds its own."""
    return (depth + 1) * (dk + 2 * depth + 8) * 2.0 ** -24


def commit_ref(inp, states, leaf, u):
    """States [B, Hv, dk, dv] after node leaf[b], and their magnitude bounds."""
    ratio = inp["Hv"] // inp["Hqk"]
    k, g, u = inp["k"].double().repeat_interleave(ratio, 1), inp["g"].double(), u.double()
    cu, parent = inp["cu"].tolist(), inp["parent"].tolist()
    out, mag = [], []
    for b in range(inp["B"]):
        path, t = [], int(leaf[b])
        while t >= 0:
            path.append(t)
            t = parent[cu[b] + t]
        S = states[int(inp["read"][b])].double()
        M = S.abs()
        for i in reversed(path):
            t = cu[b] + i
            kt, ut = k[t][:, :, None], u[t][:, None, :]
            S = decayed(inp["rule"], S, g[t]) + kt * ut
            M = decayed(inp["rule"], M, g[t].abs()) + kt.abs() * ut.abs()
        out.append(S)
        mag.append(M)
    return torch.stack(out), torch.stack(mag)


def accept_ref(cu, parent, draft, target, root):
    leaf, count, nxt = [], [], []
    for b in range(len(cu) - 1):
        at, want, n = -1, int(root[b]), 0
        while True:
            kids = [t for t in range(cu[b], cu[b + 1]) if parent[t] == at and draft[t] == want]
            if not kids:
                break
            at, want, n = kids[0] - cu[b], int(target[kids[0]]), n + 1
        leaf.append(at)
        count.append(n)
        nxt.append(want)
    return leaf, count, nxt


def beam_ref(logits, cum, finished, eos, n_out):
    """parent, token, score (FP64), finished of the best n_out, and the smallest distance of two
    neighbouring scores among the best n_out + 1 (equal scores of one beam's equal logits aside)."""
    x = logits.double().numpy().copy()
    B, K, V = x.shape
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    par, tok, sc, fin, gap = [], [], [], [], np.inf
    for b in range(B):
        s = np.full((K, V), -np.inf)
        for i in range(K):
            c = float(cum[b, i])
            if c == -np.inf:
                continue
            if finished is not None and finished[b, i]:
                s[i, eos] = c
                continue
            top = x[b, i].max()
            if top == -np.inf:
                continue
            s[i] = c + (x[b, i] - (top + np.log(np.exp(x[b, i] - top).sum())))
        flat = s.reshape(-1)
        # one beam's order is that of its logits
        order = np.lexsort((np.arange(K * V), -flat))
        best = order[:n_out + 1]
        for a, c in zip(best[:-1], best[1:]):
            if np.isfinite(flat[a]) and np.isfinite(flat[c]) and not (a // V == c // V):
                gap = min(gap, abs(flat[a] - flat[c]))
        best = best[:n_out]
        par.append(best // V)
        tok.append(best % V)
        sc.append(flat[best])
        fin.append([int((finished is not None and finished[b, i // V] != 0) or i % V == eos) for i in best])
    return np.array(par), np.array(tok), np.array(sc), np.array(fin), gap


def reorder_ref(slots, parent):
    """New slots [B][K] and the copies (source slot, destination slot)."""
    new, copies = [], []
    for row, par in zip(slots, parent):
        used, out = set(par), [None] * len(row)
        spare = [row[i] for i in range(len(row)) if i not in used]
        seen = set()
        for j, p in enumerate(par):
            if p not in seen:
                out[j] = row[p]
                seen.add(p)
            else:
                out[j] = spare.pop(0)
                copies.append((row[p], out[j]))
        new.append(out)
    return new, copies


def compact_ref(ref):
    n = len(ref)
    live = [s for s in range(n) if ref[s] > 0]
    holes = [s for s in range(len(live)) if ref[s] <= 0]
    moves = [s for s in live if s >= len(live)]
    remap = [s if ref[s] > 0 else -1 for s in range(n)]
    for s, d in zip(moves, holes):
        remap[s] = d
    new_ref = [0] * n
    for s in live:
        new_ref[remap[s]] = ref[s]
    return new_ref, remap, moves, [len(live), len(moves)]
