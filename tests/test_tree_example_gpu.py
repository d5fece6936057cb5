"""A tree of drafts run through the example's model (block and attention layers, sampling, acceptance,
commit, truncation): every node has the logits of reading its path at once, and so has what is
decoded afterwards. Bound: as for the serving test, 2e-3 on logits of unit scale."""
import pytest

from tests.test_hybrid_example_gpu import BOUND, example, ints  # noqa: F401
from tests.tree_cases import path_to

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_trees_equal_reading_their_paths(example):  # noqa: F811
    server = example.Server(seed=5)
    vocab = server.embedding.shape[0]
    lengths, slots = [1, 100, 33], [3, 0, 9]
    texts = [torch.randint(vocab, (m,), device="cuda") for m in lengths]
    server.prompt(ints(*slots), torch.cat(texts), lengths)
    trees = [[-1, 0, 0, 1, 1, 2, 5, 3, 6, 8], [-1, 0, 1, 2, 3, 4, 5, 6, 7, 8], [-1, 0, 0, 0, 1, -2, -2, -2, -2, -2]]
    m = len(trees[0])
    parents = ints(*sum(trees, [])).view(3, m)

    def alone(x, tokens):
        """Logits of reading tokens behind sequence x's text, in a slot of its own."""
        server.fork(ints(slots[x]), ints(30))
        logits = server.prompt(ints(30), tokens, [tokens.numel()])
        server.release(ints(30))
        return logits

    for step in range(3):
        tokens = torch.randint(vocab, (3, m), device="cuda", dtype=torch.int32)
        u = torch.rand(3, m, device="cuda")
        settings = dict(temperature=torch.tensor([0.0, 1.0, 0.7], device="cuda"),
                        top_p=torch.tensor([1.0, 0.9, 1.0], device="cuda"))
        # the drafts along one path of every tree agree with what is sampled: found by reading
        # ahead with the same numbers
        goal = [[0, 2, 5, 6, 8], [0, 1, 2], [0, 3]]
        for i in range(1, max(map(len, goal))):
            for x in range(3):
                if i < len(goal[x]):
                    read = alone(x, tokens[x, goal[x][:i]])
                    mine = {k: v[x:x + 1].contiguous() for k, v in settings.items()}
                    tokens[x, goal[x][i]] = server.sample(read[-1:], u[x, goal[x][i - 1]].view(1), **mine)[0]
        seen = {}
        for x, tree in enumerate(trees):
            for i in range(m):
                if tree[i] > -2:
                    seen[x, i] = alone(x, tokens[x, path_to(tree, i)])[-1]
        logits, path, kept, following = server.verify_tree(ints(*slots), tokens, parents, u, **settings)
        for (x, i), want in seen.items():
            off = (logits[x, i] - want).abs().max().item()
            assert off <= BOUND, f"step {step}, sequence {x}, node {i}: off by {off:.1e}"
        for x in range(3):
            n = kept[x].item()
            assert path[x, :len(goal[x])].tolist() == goal[x] and n >= len(goal[x])
            texts[x] = torch.cat([texts[x], tokens[x, path[x, :n].long()]])
        assert server.cache.lens[ints(*slots).long()].tolist() == [t.numel() for t in texts]
        # what is decoded next sees the accepted path and nothing else
        after = server.decode(ints(*slots), following)
        for x in range(3):
            texts[x] = torch.cat([texts[x], following[x:x + 1]])
            server.prompt(ints(31), texts[x], [texts[x].numel()])
            server.release(ints(31))
            want = read_at_once(server, texts[x])
            assert (after[x] - want).abs().max().item() <= BOUND, f"step {step}, sequence {x}"
    server.check()


def read_at_once(server, text):
    logits = server.prompt(ints(29), text, [text.numel()])[-1]
    server.release(ints(29))
    return logits


def test_the_example_runs(example):  # noqa: F811
    example.main()
