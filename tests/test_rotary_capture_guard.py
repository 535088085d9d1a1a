"""apply_rotary's refusal of a captured backward beside a living graph of another stream, on the CPU: streams, the
capture and the rotation itself are stand-ins, the graphs are PyTorch's own."""
import gc

import pytest

torch = pytest.importorskip("torch")

from exact_attention_28_gb300 import ops  # noqa: E402

POS = torch.arange(6, dtype=torch.int32)


class Streams:
    current, capturing = 0, False

    def on(self, stream, capturing=False):
        self.current, self.capturing = stream, capturing


@pytest.fixture
def streams(monkeypatch):
    gc.collect()
    s = Streams()
    monkeypatch.setattr(ops, "_raw_stream", lambda dev: s.current)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: s.capturing)
    monkeypatch.setattr(ops, "fa_rope", lambda q, k, *a, **kw: (q * 2, None if k is None else k * 2))
    return s


def leaf_of(shape=(1, 4, 6, 64)):
    return torch.zeros(shape, requires_grad=True)


def projected(x):
    return (torch.ones(1, 4, 6, 8) @ x).relu()


FORMS = {"itself": lambda x: x, "a slice": lambda x: x[:, :2], "transposed": lambda x: x.transpose(1, 2),
         "expanded": lambda x: x.expand(3, 4, 6, 64), "a view of a view": lambda x: x[:, 1:].transpose(2, 1)[:, :3]}


def grad(y, leaf):
    return torch.autograd.grad(y, leaf, torch.ones_like(y))


def rotated(x):
    return ops.apply_rotary(x, None, POS, None)


@pytest.mark.parametrize("captured", FORMS)
@pytest.mark.parametrize("eager", FORMS)
def test_refused_beside_an_eager_rotation_of_the_same_leaf(streams, eager, captured):
    leaf = leaf_of()
    kept = rotated(FORMS[eager](leaf))
    streams.on(7, capturing=True)
    y = rotated(FORMS[captured](leaf))                  # the forward alone may be captured
    with pytest.raises(RuntimeError, match="captured"):
        grad(y, leaf)
    streams.on(0)
    assert grad(kept, leaf)[0].abs().sum() > 0          # the eager graph still works
    del kept, y
    streams.on(7, capturing=True)
    grad(rotated(FORMS[captured](leaf)), leaf)          # and with it gone, so does the capture


def test_refused_behind_a_projection(streams):
    weight = leaf_of((1, 4, 8, 64))
    kept = rotated(projected(weight))
    streams.on(7, capturing=True)
    y = rotated(projected(weight))
    with pytest.raises(RuntimeError, match="captured"):
        grad(y, weight)
    del kept
    grad(y, weight)
    q, k = ops.apply_rotary(leaf_of(), projected(weight), POS, None)
    streams.on(9, capturing=True)
    with pytest.raises(RuntimeError, match="captured"):  # the other graph's k
        grad(rotated(weight.transpose(1, 2)), weight)
    del q, k


def test_other_leaves_and_the_same_stream_are_no_matter(streams):
    leaf, other = leaf_of(), leaf_of()
    kept = rotated(other[:, :2])                        # another leaf, on the default stream
    streams.on(7)
    warm = rotated(leaf[:, :2])
    del kept
    kept = None
    grad(warm, leaf)
    del warm
    streams.on(0)
    kept = rotated(other[:, :2])
    streams.on(7, capturing=True)
    first = rotated(leaf[:, :2])                        # two captures on one stream, the first one's outputs kept
    grad(first, leaf)
    grad(rotated(leaf.transpose(1, 2)), leaf)
    assert kept is not None


def test_a_node_outlives_the_rotation_that_it_was_made_for(streams):
    # the leaf's node is the default stream's: a later graph of the capture's own stream kept it alive
    leaf = leaf_of()
    first = rotated(leaf[:, :2])
    streams.on(7)
    second = rotated(leaf[:, 2:])
    del first
    streams.on(7, capturing=True)
    with pytest.raises(RuntimeError, match="captured"):
        grad(rotated(leaf[:, :2]), leaf)
    del second
    grad(rotated(leaf[:, :2]), leaf)
    # and so did a graph of another function, where the leaf itself was turned
    streams.on(0)
    first = rotated(leaf)
    other = leaf * 3
    del first
    streams.on(7, capturing=True)
    with pytest.raises(RuntimeError, match="captured"):
        grad(rotated(leaf[:, :2]), leaf)
    del other


def test_trails_go_with_their_graphs(streams):
    count = lambda: sum(len(live) for live in ops._trails.get(-1, {}).values())
    before, leaf = count(), leaf_of()
    y = [rotated(leaf[:, :2]) for _ in range(5)]
    assert count() == before + 5
    del y
    assert count() == before
    rotated(torch.zeros(1, 2, 6, 64))                   # nothing to differentiate
    assert count() == before


def test_trails_from_several_threads(streams):
    import threading
    leaf, wrong = leaf_of(), []

    def work():
        try:
            for _ in range(300):
                grad(rotated(leaf[:, :2]), leaf)
        except Exception as e:      # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for i in range(300):            # another stream's rotations, and captures, at the same time
        streams.on(i % 3)
        y = rotated(leaf_of())
        ops._meets(ops._leave_trail(y.grad_fn.next_functions, -1))
    for t in threads:
        t.join()
    assert not wrong
