"""Refusals of the serving operators' host checks (fake, never dereferenced device addresses; no
call in this file reaches a kernel launch), and the plain implementations against one another."""
import ctypes
import os

import numpy as np
import pytest
import torch

import serving_ref as R
from gated_deltanet_recurrent_la_b200 import lastate as L

A = 0x7f0000000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from gated_deltanet_recurrent_la_b200 import build
        build.build()
    return L.lib()


def pool(dtype=1, n=8, shape=(2, 4, 128, 128), data=A, n_hp=0, mask=None):
    return L.la_pool(ctypes.c_void_p(data), dtype, n, L.la_shape(*shape), n_hp, mask)


def tree(lib, rule=3, src=None, read=None, n=4, cu=A, T=10, parent=A, m=16, q=A, k=A, v=A, io=1, g=A, beta=A, o=A, u=A, err=A):
    src = src or pool()
    return lib.la_state_tree(rule, ctypes.byref(src), read, n, cu, T, parent, m, q, k, v, io, g, beta, 1.0, o, u, err, None)


def test_tree_host_errors(lib):
    assert tree(lib, n=0) == L.LA_OK
    for bad in (dict(rule=5), dict(rule=-1), dict(m=65), dict(io=2), dict(src=pool(shape=(2, 4, 32, 32))), dict(src=pool(dtype=7))):
        assert tree(lib, **bad) == L.LA_ERR_UNSUPPORTED, bad
    for bad in (dict(err=None), dict(cu=None), dict(parent=None), dict(q=None), dict(k=None), dict(v=None), dict(o=None),
                dict(g=None), dict(beta=None), dict(src=pool(data=0)), dict(rule=4, g=None),
                dict(src=pool(dtype=2, n_hp=16))):
        assert tree(lib, **bad) == L.LA_ERR_NULL, bad
    for bad in (dict(n=-1), dict(T=-1), dict(m=0), dict(n=9), dict(src=pool(shape=(3, 4, 128, 128))), dict(n=1 << 30, read=A)):
        assert tree(lib, **bad) == L.LA_ERR_SHAPE, bad
    for bad in (dict(q=A + 8), dict(k=A + 2), dict(v=A + 4), dict(o=A + 8), dict(u=A + 4), dict(cu=A + 2), dict(parent=A + 1),
                dict(read=A + 2), dict(err=A + 1), dict(beta=A + 2), dict(rule=4, g=A + 4)):
        assert tree(lib, **bad) == L.LA_ERR_ALIGN, bad


def accept(lib, n=3, cu=A, T=5, parent=A, m=8, draft=A, target=A, root=A, leaf=A, count=A, nxt=A, err=A):
    return lib.la_tree_accept(n, cu, T, parent, m, draft, target, root, leaf, count, nxt, err, None)


def test_accept_host_errors(lib):
    assert accept(lib, n=0) == L.LA_OK
    for name in ("cu", "parent", "draft", "target", "root", "leaf", "count", "nxt", "err"):
        assert accept(lib, **{name: None}) == L.LA_ERR_NULL, name
        assert accept(lib, **{name: A + 2}) == L.LA_ERR_ALIGN, name
    assert accept(lib, n=-1) == accept(lib, T=-1) == accept(lib, m=0) == L.LA_ERR_SHAPE
    assert accept(lib, m=65) == L.LA_ERR_UNSUPPORTED


def commit(lib, rule=3, src=None, read=None, dst=None, write=None, n=4, cu=A, T=10, parent=A, leaf=A, m=16, k=A, io=1, g=A,
           u=A, err=A):
    src = src or pool()
    dst = dst or src
    return lib.la_state_tree_commit(rule, ctypes.byref(src), read, ctypes.byref(dst), write, n, cu, T, parent, leaf, m, k, io,
                                    g, u, err, None)


def test_commit_host_errors(lib):
    assert commit(lib, n=0) == L.LA_OK
    for bad in (dict(rule=9), dict(m=65), dict(io=2), dict(dst=pool(dtype=0)), dict(src=pool(shape=(2, 4, 128, 32)),
                                                                                    dst=pool(shape=(2, 4, 128, 32)))):
        assert commit(lib, **bad) == L.LA_ERR_UNSUPPORTED, bad
    for name in ("cu", "parent", "leaf", "k", "u", "g", "err"):
        assert commit(lib, **{name: None}) == L.LA_ERR_NULL, name
    for bad in (dict(n=-1), dict(m=0), dict(n=9), dict(n=9, read=A), dict(n=9, write=A), dict(dst=pool(shape=(2, 4, 128, 64))),
                dict(src=pool(dtype=2, n_hp=16, mask=A), dst=pool(dtype=2, n_hp=8, mask=A, data=A + 4096))):
        assert commit(lib, **bad) == L.LA_ERR_SHAPE, bad
    for name in ("cu", "parent", "leaf", "k", "u", "err", "read", "write"):
        assert commit(lib, **{name: A + 2}) == L.LA_ERR_ALIGN, name
    two = dict(src=pool(dtype=2, n_hp=16, mask=A), dst=pool(dtype=2, n_hp=16, mask=A + 64))
    assert commit(lib, **two) == L.LA_ERR_ALIAS


def beam(lib, n=2, K=4, V=100, x=A, io=1, stride=100, cum=A, fin=A, eos=3, n_out=4, par=A, tok=A, sc=A, fo=A, ws=A, nws=1 << 20):
    return lib.la_beam_select(n, K, V, x, io, stride, cum, fin, eos, n_out, par, tok, sc, fo, ws, nws, None)


def test_beam_host_errors(lib):
    assert beam(lib, n=0) == L.LA_OK
    for bad in (dict(n=-1), dict(K=0), dict(V=0), dict(n_out=0), dict(stride=99), dict(eos=-1), dict(eos=100), dict(nws=8),
                dict(K=1, V=3, stride=3, eos=2, n_out=4), dict(n=1 << 30)):
        assert beam(lib, **bad) == L.LA_ERR_SHAPE, bad
    for bad in (dict(K=65), dict(n_out=65), dict(io=2)):
        assert beam(lib, **bad) == L.LA_ERR_UNSUPPORTED, bad
    for name in ("x", "cum", "par", "tok", "sc", "ws"):
        assert beam(lib, **{name: None}) == L.LA_ERR_NULL, name
    for bad in (dict(x=A + 1), dict(io=0, x=A + 2), dict(cum=A + 2), dict(fin=A + 2), dict(par=A + 2), dict(tok=A + 2),
                dict(sc=A + 2), dict(fo=A + 2), dict(ws=A + 8)):
        assert beam(lib, **bad) == L.LA_ERR_ALIGN, bad
    assert L.la_beam_workspace_bytes(0, 65, 10, 1) == 0 and L.la_beam_workspace_bytes(2, 4, 100, 4) > 0


def slab_array(*slabs):
    return (L.la_slab * len(slabs))(*slabs)


GOOD = (L.la_slab(A, 64, 8), L.la_slab(A + 4096, 32, 8))


def test_slab_host_errors(lib):
    def reorder(slabs=GOOD, n=None, B=2, K=3, slots=A, par=A + 64, new=A + 128, err=A):
        arr = None if slabs is None else slab_array(*slabs)
        return lib.la_state_pool_reorder(arr, len(slabs or ()) if n is None else n, B, K, slots, par, new, err, None)

    assert reorder(B=0) == L.LA_OK
    assert reorder(slabs=None, n=1) == L.LA_ERR_NULL
    assert reorder(n=0) == L.LA_ERR_SHAPE
    assert reorder(slabs=(L.la_slab(A, 64, 8),) * 129) == L.LA_ERR_UNSUPPORTED
    assert reorder(slabs=(L.la_slab(A, 64, 8), L.la_slab(A, 64, 9))) == L.LA_ERR_SHAPE
    assert reorder(slabs=(L.la_slab(A, 40, 8),)) == reorder(slabs=(L.la_slab(A, 0, 8),)) == L.LA_ERR_SHAPE
    assert reorder(slabs=(L.la_slab(None, 64, 8),)) == L.LA_ERR_NULL
    assert reorder(slabs=(L.la_slab(A + 8, 64, 8),)) == L.LA_ERR_ALIGN
    assert reorder(K=65) == L.LA_ERR_UNSUPPORTED
    assert reorder(B=-1) == reorder(K=0) == L.LA_ERR_SHAPE
    for name in ("slots", "par", "new", "err"):
        assert reorder(**{name: None}) == L.LA_ERR_NULL
        assert reorder(**{name: A + 2}) == L.LA_ERR_ALIGN
    assert reorder(new=A) == reorder(new=A + 64) == L.LA_ERR_ALIAS

    def fork(ref=A, n=3, src=A + 64, new=A + 128, err=A):
        return lib.la_state_pool_fork(slab_array(*GOOD), 2, ref, n, src, new, err, None)

    assert fork(n=0) == L.LA_OK
    assert fork(n=-1) == L.LA_ERR_SHAPE
    for name in ("ref", "src", "new", "err"):
        assert fork(**{name: None}) == L.LA_ERR_NULL
        assert fork(**{name: A + 2}) == L.LA_ERR_ALIGN
    assert fork(new=A + 64) == fork(src=A) == fork(new=A) == L.LA_ERR_ALIAS

    for fn in (lib.la_state_pool_alloc, lib.la_state_pool_share, lib.la_state_pool_free):
        assert fn(A, 8, 0, A + 64, A, None) == L.LA_OK
        assert fn(A, 8, -1, A + 64, A, None) == fn(A, -1, 1, A + 64, A, None) == L.LA_ERR_SHAPE
        assert fn(None, 8, 2, A + 64, A, None) == fn(A, 8, 2, None, A, None) == fn(A, 8, 2, A + 64, None, None) == L.LA_ERR_NULL
        assert fn(A + 2, 8, 2, A + 64, A, None) == fn(A, 8, 2, A + 65, A, None) == L.LA_ERR_ALIGN
        assert fn(A, 8, 2, A, A, None) == L.LA_ERR_ALIAS

    def compact(*ptrs, err=A):
        return lib.la_state_pool_compact(slab_array(*GOOD), 2, *ptrs, err, None)

    good = [A, A + 64, A + 128, A + 192, A + 256]
    assert compact(*good, err=None) == L.LA_ERR_NULL
    for i in range(5):
        assert compact(*good[:i], None, *good[i + 1:]) == L.LA_ERR_NULL
        assert compact(*good[:i], good[i] + 2, *good[i + 1:]) == L.LA_ERR_ALIGN
        assert compact(*good[:i], good[i - 1], *good[i + 1:]) == L.LA_ERR_ALIAS

    def remap(n=3, table=A, slots=8, rm=A + 64, new=A, err=A):
        return lib.la_state_pool_remap(n, table, slots, rm, new, err, None)

    assert remap(n=0) == L.LA_OK
    assert remap(n=-1) == remap(slots=-1) == remap(n=1 << 31) == L.LA_ERR_SHAPE
    for name in ("table", "rm", "new", "err"):
        assert remap(**{name: None}) == L.LA_ERR_NULL
        assert remap(**{name: A + 2}) == L.LA_ERR_ALIGN
    assert remap(new=A + 64) == L.LA_ERR_ALIAS
    s = L.la_slab()
    p = pool()
    assert lib.la_pool_slab(ctypes.byref(p), ctypes.byref(s)) == L.LA_OK
    assert (s.data, s.slot_bytes, s.n_slots) == (A, 4 * 128 * 128 * 2, 8)
    assert lib.la_pool_slab(ctypes.byref(p), None) == L.LA_ERR_NULL


@pytest.mark.parametrize("rule", R.RULES)
def test_plain_tree_is_the_oracle_scan_along_every_path(rule, orc):
    """A node's output is the last output of the token-serial scan over its path, and its
    commit that scan's final state (the oracle shares no code with the plain tree)."""
    inp = R.tree_inputs(lens=[9], Hqk=1, Hv=2, dk=16, dv=16, rule=rule, state_dtype=torch.float32, io_dtype=torch.float32, seed=4)
    o, u, _, _, _ = R.tree_ref(inp, inp["pool"])
    n64 = lambda x: x.double().numpy()  # noqa: E731
    for leaf in range(9):
        path, t = [], leaf
        while t >= 0:
            path.insert(0, t)
            t = int(inp["parent"][t])
        S, os_, _ = orc.scan(rule, 1, np.array([0, len(path)], np.int32), n64(inp["q"][path]), n64(inp["k"][path]),
                             n64(inp["v"][path]), n64(inp["g"][path]) if R.uses_gate(rule) else None,
                             n64(inp["beta"][path]) if R.uses_beta(rule) else None, inp["scale"],
                             src_pool=n64(inp["pool"]), read_slot=inp["read"].numpy(), dst_dtype="f64", io_dtype="f64")
        np.testing.assert_allclose(o[leaf].numpy(), os_[-1], rtol=0, atol=1e-12)
        state, _ = R.commit_ref(inp, inp["pool"], [leaf], u)
        np.testing.assert_allclose(state.numpy(), S, rtol=0, atol=1e-12)


def test_tree_rows_beyond_32_bit_offsets_are_refused(lib):
    """64 rows of all value heads have to fit 32-bit element offsets."""
    assert tree(lib, n=1, src=pool(shape=(1, 1 << 19, 128, 128))) == L.LA_ERR_SHAPE
