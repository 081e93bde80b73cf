"""Refusals of the serving operators that keep their kernels within the caller's arrays (fake,
never dereferenced device addresses; no call in this file may reach a kernel launch)."""
import os

import pytest

from gated_deltanet_recurrent_la_b200 import lastate as L

A = 0x7f0000000000
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from gated_deltanet_recurrent_la_b200 import build
        build.build()
    return L.lib()


def beam(lib, n=2, K=4, V=100, x=A, io=1, stride=100, cum=A + MB, fin=A + 2 * MB, eos=3, n_out=4, par=A + 3 * MB, tok=A + 4 * MB,
         sc=A + 5 * MB, fo=A + 6 * MB, ws=A + 7 * MB, nws=MB):
    return lib.la_beam_select(n, K, V, x, io, stride, cum, fin, eos, n_out, par, tok, sc, fo, ws, nws, None)


def test_beam_arrays_that_overlap(lib):
    """In place only where a sequence's outputs lie on its own inputs."""
    for n_out in (3, 5):  # of four beams
        assert beam(lib, n_out=n_out, sc=A + MB) == L.LA_ERR_ALIAS
        assert beam(lib, n_out=n_out, fo=A + 2 * MB) == L.LA_ERR_ALIAS
    assert beam(lib, sc=A + MB + 4) == beam(lib, fo=A + 2 * MB - 4) == L.LA_ERR_ALIAS  # shifted by one
    assert beam(lib, sc=A + 2 * MB) == beam(lib, fo=A + MB) == L.LA_ERR_ALIAS          # the other's input
    for name in ("par", "tok"):
        assert beam(lib, **{name: A + MB}) == beam(lib, **{name: A + 2 * MB}) == L.LA_ERR_ALIAS
    names, at = ("par", "tok", "sc", "fo"), [A + 3 * MB, A + 4 * MB, A + 5 * MB, A + 6 * MB]
    for i, name in enumerate(names):
        for j in range(4):
            if j != i:
                assert beam(lib, **{name: at[j] + 28}) == L.LA_ERR_ALIAS, (name, j)
        assert beam(lib, **{name: A + 7 * MB + 8}) == L.LA_ERR_ALIAS                    # the workspace
    assert beam(lib, ws=A + 64) == beam(lib, ws=A + MB) == beam(lib, ws=A + 2 * MB) == L.LA_ERR_ALIAS


TOO_MANY = (1 << 31) - 65536  # one above the largest count


def test_counts_that_32_bit_counters_would_pass(lib):
    """Loops step past the end of a row or a list; near 2^31 their counters would wrap."""
    big = 1 << 62
    for n in (TOO_MANY, (1 << 31) - 1):
        assert beam(lib, V=n, stride=n, ws=big, nws=1 << 40) == L.LA_ERR_SHAPE
        assert L.la_beam_workspace_bytes(2, 4, n, 4) == 0
        for fn in (lib.la_state_pool_alloc, lib.la_state_pool_share, lib.la_state_pool_free):
            assert fn(A, 8, n, A + MB, A, None) == fn(A, n, 8, A + MB, A, None) == L.LA_ERR_SHAPE
        slabs = (L.la_slab * 1)(L.la_slab(A, 16, 8))
        assert lib.la_state_pool_fork(slabs, 1, A, n, A + MB, A + 2 * MB, A, None) == L.LA_ERR_SHAPE
        slabs = (L.la_slab * 1)(L.la_slab(A, 16, n))
        assert lib.la_state_pool_fork(slabs, 1, A, 3, A + MB, A + 2 * MB, A, None) == L.LA_ERR_SHAPE
        assert lib.la_state_pool_compact(slabs, 1, A, A + MB, A + 2 * MB, A + 3 * MB, A + 4 * MB, A, None) == L.LA_ERR_SHAPE
        assert lib.la_state_pool_reorder(slabs, 1, 2, 3, A, A + MB, A + 2 * MB, A, None) == L.LA_ERR_SHAPE


def test_lists_of_slots_that_overlap(lib):
    """By a few entries, where both arrays are written or read by many threads at once."""
    slabs = (L.la_slab * 1)(L.la_slab(A, 16, 8))
    B = A + MB
    for d in (-20, -4, 4, 20):  # 6 beams: 24 bytes
        assert lib.la_state_pool_reorder(slabs, 1, 2, 3, B, B + 512, B + d, A, None) == L.LA_ERR_ALIAS
        assert lib.la_state_pool_reorder(slabs, 1, 2, 3, B + 512, B, B + d, A, None) == L.LA_ERR_ALIAS
    for fn in (lib.la_state_pool_alloc, lib.la_state_pool_share, lib.la_state_pool_free):  # 8 counts, 3 slots
        assert [fn(B, 8, 3, B + d, A, None) for d in (-8, 4, 28)] == [L.LA_ERR_ALIAS] * 3
    assert lib.la_state_pool_fork(slabs, 1, B, 3, B + 64, B + 72, A, None) == L.LA_ERR_ALIAS
    assert lib.la_state_pool_fork(slabs, 1, B, 3, B + 28, B + 72, A, None) == L.LA_ERR_ALIAS
    assert lib.la_state_pool_fork(slabs, 1, B, 3, B + 72, B + 28, A, None) == L.LA_ERR_ALIAS
    good = [B, B + 64, B + 128, B + 192, B + 256]  # 8 slots: 32 bytes, and the counts
    for i in range(5):
        for j in range(5):
            if j != i:
                ptrs = [good[j] + 4 if k == i else p for k, p in enumerate(good)]
                assert lib.la_state_pool_compact(slabs, 1, *ptrs, A, None) == L.LA_ERR_ALIAS, (i, j)
    assert lib.la_state_pool_remap(5, B, 8, B + 64, B + 4, A, None) == L.LA_ERR_ALIAS
    assert lib.la_state_pool_remap(5, B, 8, B + 64, B + 48, A, None) == L.LA_ERR_ALIAS


def test_empty_lists_overlap_nothing(lib):
    for fn in (lib.la_state_pool_alloc, lib.la_state_pool_share, lib.la_state_pool_free):
        assert fn(A, 8, 0, A + 8, A, None) == L.LA_OK
