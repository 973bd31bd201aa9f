"""Trees of new tokens for the tests: random ones of several shapes, and their paths, plainly."""
import random


def path(parents, i):
    """The nodes from a root to i."""
    out = []
    while i >= 0:
        out.append(i)
        i = parents[i]
    return out[::-1]


def random_tree(n, shape, seed):
    """Parents of n nodes.  chain: one after another; star: all from the context; bush: any earlier node;
    levels: a few nodes to a level; forest: several roots, recent parents."""
    r = random.Random(seed * 1000 + n)
    if shape == "chain":
        return list(range(-1, n - 1))
    if shape == "star":
        return [-1] * n
    if shape == "bush":
        return [r.randint(-1, i - 1) for i in range(n)]
    if shape == "levels":
        w = max(1, n // 6)
        return [-1 if i < w else r.randrange((i // w - 1) * w, (i // w) * w) for i in range(n)]
    return [r.randint(max(-1, i - 5), i - 1) if i and r.random() < 0.9 else -1 for i in range(n)]


SHAPES = ["chain", "star", "bush", "levels", "forest"]


def sees(parents, c, window, sinks):
    """For each node the places of the cache that it sees, as a set: the definition."""
    depth = [len(path(parents, i)) - 1 for i in range(len(parents))]
    out = []
    for i in range(len(parents)):
        p = c + depth[i]
        keys = [(t, t) for t in range(max(c, 0))] + [(c + j, c + depth[j]) for j in path(parents, i)]
        out.append({place for place, pos in keys if place >= 0 and (not window or pos > p - window or pos < sinks)})
    return out
