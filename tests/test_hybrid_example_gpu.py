"""The example's model served step by step (prompts, chunks, forks, single tokens, drafts and
their rollback, compaction) gives the logits of reading every sequence in at once.

Bound: both sides compute in fp32 through the same layers, with sums in other orders. A layer
is held to 1e-4 of its outputs' unit scale by its own tests; four layers in a row, each at
most doubling what comes in (their inputs are normalised to unit scale), and the logits'
product make 1e-4 * (1 + 2 + 4 + 8) < 2e-3 on logits of unit scale."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BOUND = 2e-3


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "hybrid_serving.py")
    spec = importlib.util.spec_from_file_location("hybrid_serving", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def ints(*x):
    return torch.tensor(x, device="cuda", dtype=torch.int32)


def test_serving_equals_reading_at_once(example):
    server = example.Server(seed=3)
    vocab = server.embedding.shape[0]
    lengths = [1, 150, 37, 64]
    slots, twins = [3, 0, 9, 17], [4, 1, 10, 18]
    texts, seen = {s: [] for s in slots + twins}, {s: [] for s in slots + twins}

    def note(some, tokens, logits):
        for i, s in enumerate(some):
            texts[s].append(tokens[i].flatten())
            seen[s].append(logits[i].reshape(-1, vocab))

    def read(sizes):
        tokens = torch.randint(vocab, (sum(sizes),), device="cuda")
        logits = server.prompt(ints(*slots), tokens, sizes)
        note(slots, tokens.split(sizes), logits.split(sizes))

    read(lengths)
    read([20, 0, 1, 30])  # a second chunk of the prompts
    server.fork(ints(*slots), ints(*twins))
    for s, t in zip(slots, twins):
        texts[t], seen[t] = list(texts[s]), list(seen[s])
    everyone = slots + twins
    for _ in range(5):
        tokens = torch.randint(vocab, (len(everyone),), device="cuda")
        note(everyone, tokens, server.decode(ints(*everyone), tokens))
    # drafts of 4: kept are those that agree with the model, whose choice after the first token
    # is found on a fork that is thrown away
    tokens = torch.randint(vocab, (len(everyone), 4), device="cuda")
    probe = [s + 12 if s != 17 else 31 for s in slots]  # forks of the first four
    server.fork(ints(*slots), ints(*probe))
    tokens[:4, 1] = server.decode(ints(*probe), tokens[:4, 0]).argmax(-1)
    server.release(ints(*probe))
    logits, kept = server.verify(ints(*everyone), tokens)
    kept = kept.tolist()
    assert min(kept[:4]) >= 2
    note(everyone, [tokens[i, :n] for i, n in enumerate(kept)],
         [logits[i, :n] for i, n in enumerate(kept)])
    server.release(ints(*slots))
    server.cache.compact()
    for _ in range(3):
        tokens = torch.randint(vocab, (len(twins),), device="cuda")
        note(twins, tokens, server.decode(ints(*twins), tokens))
    server.check()
    assert server.cache.lens[ints(*twins).long()].tolist() == [sum(map(len, texts[t])) for t in twins]
    server.release(ints(*twins))
    assert (server.cache.refs == 0).all() and (server.cache.lens == 0).all()

    whole = [torch.cat(texts[s]) for s in everyone]
    sizes = [len(t) for t in whole]
    ref = server.prompt(ints(*everyone), torch.cat(whole), sizes).split(sizes)
    server.check()
    for s, r in zip(everyone, ref):
        assert (torch.cat(seen[s]) - r).abs().max().item() <= BOUND, f"slot {s}"


def test_main_runs(example, capsys):
    example.main()
    assert "pages in use" in capsys.readouterr().out
