"""The example's model: caches written by chunks, by single tokens and by accepted tree paths hold the same values."""
import os
import sys

import pytest

from pace_testlib import ensure_built

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def E():
    ensure_built()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import hybrid_layers
    return hybrid_layers


def held(stack, n):
    import torch
    kv = stack.layers[0][0]
    k, v = torch.empty(2, stack.B, n, stack.kv_heads, stack.d, dtype=torch.bfloat16, device="cuda")
    kv.read(k, v, stack.table, end=stack.lens)
    return k, v


def test_example_runs(E):
    model, plain, tree, want, got, mean = E.main()
    assert plain.status() == tree.status() == model.status() == [0]
    assert want.shape == got.shape == (4, 64)
    assert mean > 1.5


def test_caches_agree_however_they_were_written(E):
    """One attention layer: keys and values depend on the tokens alone, so that chunks, single tokens and kept tree paths have to
    leave the same codes."""
    import torch
    B, vocab = 3, 512
    g = torch.Generator(device="cuda").manual_seed(5)
    tokens = torch.randint(0, vocab, (B, 300), generator=g, device="cuda")
    chunks, single, tree = (E.Stack(["attend"], B, 512) for _ in range(3))
    chunks.prompt(tokens)
    for t in range(300):
        single.forward(tokens[:, t:t + 1])
        single.lens += 1
    # trees of seven nodes around the wanted path: nodes 0, 2 and 5 hold its next three tokens
    parents = [0, 0, 0, 1, 2, 2, 4]
    see = torch.zeros(7, 7, dtype=torch.bool)
    depth = [0] * 7
    for i, p in enumerate(parents):
        if i:
            see[i], depth[i] = see[p], depth[p] + 1
        see[i, i] = True
    words = torch.tensor([[sum(1 << j for j in range(7) if see[i, j])] for i in range(7)], dtype=torch.int32, device="cuda")
    idx = torch.tensor([[0, 2, 5]] * B, dtype=torch.int32, device="cuda")
    for t in range(0, 300, 3):
        nodes = torch.randint(0, vocab, (B, 7), generator=g, device="cuda")
        for node, at in ((0, t), (2, t + 1), (5, t + 2)):
            nodes[:, node] = tokens[:, at]
        tree.forward(nodes, positions=tree.lens[:, None] + torch.tensor(depth, dtype=torch.int32, device="cuda"),
                     mask=words.expand(B, 7, 1).contiguous())
        tree.layers[0][0].keep(tree.lens, tree.table, idx, torch.full((B,), 3, dtype=torch.int32, device="cuda"))
        tree.lens += 3
    a, b, c = (held(s, 300) for s in (chunks, single, tree))
    for x, y, z in zip(a, b, c):
        assert torch.isfinite(x).all()
        # the projections are library products of other shapes, which may round an element the other way: at most a code, in few places
        for other in (y, z):
            assert (x != other).float().mean() < 0.01 and (x - other).abs().max() <= 0.26 * x.abs().max()


def test_drafts_are_refused_beside_recurrent_layers(E):
    import torch
    model = E.Stack(["delta", "attend"], 1, 64)
    with pytest.raises(ValueError):
        model.generate_drafted(torch.zeros(1, dtype=torch.int64, device="cuda"), 1, None, [0])
