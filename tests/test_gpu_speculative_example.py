"""The speculative example runs, keeps its books, and samples as the target does when its drafts are as good as none."""
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
    import speculative_sampling
    return speculative_sampling


def test_example_runs(E):
    server, out, mean, held = E.main(steps=10)
    assert server.status() == [0, 0, 0, 0]
    assert all(len(o) >= 10 and all(0 <= t < server.vocab for t in o) for o in out)
    assert 1 <= mean <= 5                                    # (a path of four drafts and the next token)
    lens = server.lens.tolist()
    assert [n > 0 for n in lens] == [True, False, False, False, True, False, False, False]
    assert held == sum(-(-n // E.PAGE) for n in lens) == int((server.table >= 0).sum())


def test_samples_that_share_pages_do_not_touch_one_another(E):
    """Two rows forked from one prompt go on with different tokens: each holds what a row of its own would."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(2)
    prompt = torch.randint(0, 512, (90,), generator=g, device="cuda").tolist()
    forked, alone = E.Server(["delta", "attend"], 2, 512), E.Server(["delta", "attend"], 2, 512)
    forked.prompt([prompt, []])
    forked.fork([0, 0])
    alone.prompt([prompt, prompt])
    more = torch.randint(0, 512, (2, 12), generator=g, device="cuda", dtype=torch.int32)
    n = torch.full((2,), 12, dtype=torch.int32, device="cuda")
    for s in (forked, alone):
        s.take(n)
    a, b = forked.forward(more, n), alone.forward(more, n)
    assert torch.equal(a, b)
    assert torch.equal(forked.layers[0][1].states, alone.layers[0][1].states)


def test_a_row_given_up_begins_anew(E):
    """A prompt of one token (nothing of it goes through the layers before the first tree) in a row that another sequence has left: the samples and
    the state of a server in which the row was never used."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    old, other = (torch.randint(0, 512, (n,), generator=g, device="cuda").tolist() for n in (80, 50))
    used, fresh = E.Server(["delta", "attend"], 2, 512), E.Server(["delta", "attend"], 2, 512)
    used.prompt([old, other])
    used.fork([-1, 1])
    fresh.prompt([[], other])
    got = []
    for s in (used, fresh):
        last = s.prompt([[7], []])
        out, _ = s.sample(last, torch.tensor([True, False], device="cuda"), 6, [0, 0, 0, 1, 2], torch.Generator(device="cuda").manual_seed(4))
        got.append((out[0], s.layers[0][1].states[0].clone()))
    assert got[0][0] == got[1][0] and torch.equal(got[0][1], got[1][1])


def test_tokens_are_distributed_as_the_targets(E):
    """The token after a prompt, from trees whose drafts come from the bigrams alone: 4,096 samples have the frequencies that the target gives (each off
    by at most five times sqrt(f (1 - f) / 4096))."""
    import torch
    rows, vocab, turns = 256, 8, 16
    s, alone = E.Server(["delta", "attend"], rows, 128, vocab=vocab), E.Server(["delta", "attend"], rows, 128, vocab=vocab)
    prompt = torch.randint(0, vocab, (40,), generator=torch.Generator().manual_seed(5)).tolist()
    for x in (s, alone):
        x.prompt([prompt] + [[]] * (rows - 1))
        x.fork([0] * rows)
    one = torch.ones(rows, dtype=torch.int32, device="cuda")
    alone.take(one)
    last = torch.full((rows,), prompt[-1], dtype=torch.int32, device="cuda")
    p = torch.softmax(alone.forward(last[:, None], one)[0, 0], -1)
    q = torch.softmax(s.bigrams[prompt[-1]], -1)
    assert (p - q).abs().max() > 0.05                        # (the drafts' distribution is another)
    states, lens = s.layers[0][1].states.clone(), s.lens.clone()
    g, count = torch.Generator(device="cuda").manual_seed(6), torch.zeros(vocab, device="cuda")
    for _ in range(turns):
        out, _ = s.sample(last, torch.ones(rows, dtype=torch.bool, device="cuda"), 1, [0, 0, 0, 1], g)
        count += torch.bincount(torch.tensor([o[0] for o in out], device="cuda"), minlength=vocab)
        s.layers[0][1].states.copy_(states)
        s.lens.copy_(lens)
        s.pages.select(s.table, s.lens)
    n = rows * turns
    assert ((count / n - p).abs() <= 5 * (p * (1 - p) / n).sqrt()).all()
