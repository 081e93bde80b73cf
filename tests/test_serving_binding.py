"""The Python binding's own checks of the serving operators: arrays whose sizes the library takes
from another one's.  The library is replaced by a stub, the tensors only say that they are on a
device."""
import pytest
import torch

from gated_deltanet_recurrent_la_b200 import lastate as L


class OnDevice(torch.Tensor):
    is_cuda = True


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    """The calls that reach the library: (name, arguments)."""
    got = []

    class Stub:
        def __getattr__(self, name):
            return lambda *args: got.append((name, args)) or L.LA_OK

    monkeypatch.setattr(L, "lib", lambda: Stub())
    monkeypatch.setattr(L, "_stream", lambda stream: 0)
    return got


def z(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


def f(*shape):
    return z(*shape, dtype=torch.float32)


class FakePool:
    ref = None


class FakeSlabs:
    array, n = None, 1


ARGS = {
    "la_beam_select": dict(logits=f(2, 3, 10), cum_score=f(2, 3), finished=z(2, 3), eos_token=1, parent=z(2, 4), token=z(2, 4),
                           score=f(2, 4), finished_out=z(2, 4), workspace=z(64)),
    "la_state_pool_reorder": dict(slabs=FakeSlabs, slots=z(2, 3), parent=z(2, 3), new_slots=z(2, 3), err_word=z(1)),
    "la_state_pool_remap": dict(table=z(5), remap=z(8), new_table=z(5), err_word=z(1)),
    "la_tree_accept": dict(cu_nodes=z(4), parent=z(9), max_nodes=4, draft=z(9), target=z(9), root=z(3), leaf=z(3), count=z(3),
                           next_token=z(3), err_word=z(1)),
    "la_state_tree": dict(rule="delta", src=FakePool, read_slot=z(3), cu_nodes=z(4), parent=z(9), max_nodes=4, q=f(9, 1, 16),
                          k=f(9, 1, 16), v=f(9, 1, 16), g=None, beta=f(9, 1), scale=1.0, o=f(9, 1, 16), u=None, err_word=z(1)),
    "la_state_tree_commit": dict(rule="delta", src=FakePool, read_slot=z(3), dst=FakePool, write_slot=z(3), cu_nodes=z(4),
                                 parent=z(9), leaf=z(3), max_nodes=4, k=f(9, 1, 16), g=None, u=f(9, 1, 16), err_word=z(1)),
}
SIZED = [("la_beam_select", x) for x in ("cum_score", "finished", "parent", "token", "score", "finished_out")] + \
    [("la_state_pool_reorder", "parent"), ("la_state_pool_reorder", "new_slots"), ("la_state_pool_remap", "new_table")] + \
    [("la_tree_accept", x) for x in ("root", "leaf", "count", "next_token")] + [("la_state_tree", "read_slot")] + \
    [("la_state_tree_commit", x) for x in ("read_slot", "write_slot", "leaf")]


@pytest.mark.parametrize("call,name", SIZED)
def test_shorter_arrays_are_refused_and_longer_ones_taken(call, name, calls):
    args = ARGS[call]
    getattr(L, call)(**args)
    assert [c[0] for c in calls] == [call]
    t = args[name]
    with pytest.raises(ValueError, match="entries expected"):
        getattr(L, call)(**{**args, name: t[:-1].contiguous()})
    assert len(calls) == 1
    getattr(L, call)(**{**args, name: torch.cat([t, t])})
    assert len(calls) == 2


@pytest.mark.parametrize("call,place,names", [("la_tree_accept", 2, ("parent", "draft", "target")),
                                              ("la_state_tree", 5, ("parent", "q")), ("la_state_tree_commit", 7, ("parent", "k"))])
def test_nodes_are_counted_by_the_shortest_array(call, place, names, calls):
    args = ARGS[call]
    for name in names:
        getattr(L, call)(**{**args, name: args[name][:7].contiguous()})
        assert calls[-1][1][place] == 7
