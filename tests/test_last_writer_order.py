"""Memory order of the few-token layer's last sum (no GPU): the warp that counts the last entry of 32 output rows
reads, with all its lanes, what all lanes of other CTAs' warps stored.  The operations between the store and the
reads are taken from the kernel's source; every read has to come after every store of every other warp by

- program order of a lane from an operation to a later fence or barrier of it, and from those to what follows,
- a warp barrier (__syncwarp) between the lanes of a warp,
- the counter's atomics, from a lane with a fence before its own to a lane with a fence after its own.

A shuffle hands a value round and orders no memory."""
import itertools
import re
from pathlib import Path

import pytest

SOURCE = Path(__file__).resolve().parents[1] / "routed_expert_moe_b200" / "csrc" / "few.cu"
LANES = 3          # lane 0 and two others stand for the warp
OPS = [("store", r"__stcg\(a\.y"), ("barrier", r"__syncwarp\(\)"), ("enter0", r"if \(lane == 0\) \{"), ("leave0", r"^\s*\}\s*$"),
       ("fence", r"__threadfence\(\)"), ("count", r"atomicAdd\(summed"), ("shuffle", r"__shfl_sync\("),
       ("read", r"fl_combine\(a,")]


def kernel_operations():
    """(kind, by lane 0 alone) from the store of an entry's rows to the sum."""
    text = SOURCE.read_text()
    body = text[text.index("__stcg(a.y"):]
    body = body[:body.index("fl_combine(a,") + len("fl_combine(a,")]
    ops, alone = [], False
    for line in body.splitlines():
        line = line.split("//")[0]
        found = sorted((m.start(), kind) for kind, pat in OPS for m in re.finditer(pat, line))
        for _, kind in found:
            if kind == "enter0":
                alone = True
            elif kind == "leave0":
                alone = False
            else:
                ops.append((kind, alone))
    return ops


def unordered(ops):
    """Pairs (storing lane, reading lane) of two warps without an order, when `a` counts before `b`."""
    nodes = [(w, lane, i) for w in "ab" for i, (_, alone) in enumerate(ops) for lane in range(1 if alone else LANES)]
    after = {n: set() for n in nodes}
    strong = {"fence", "barrier"}
    for (w, l, i), (v, m, j) in itertools.product(nodes, nodes):
        k, kk = ops[i][0], ops[j][0]
        if w == v and l == m and i < j and (k in strong or kk in strong):
            after[w, l, i].add((v, m, j))
        if w == v and i == j and l != m and k == "barrier":
            # all lanes' earlier operations come before all lanes' later ones
            for j2 in range(i + 1, len(ops)):
                if (w, m, j2) in after:
                    after[w, l, i].add((w, m, j2))
        if (w, v) == ("a", "b") and k == kk == "count" and i == j:
            fenced = any(o == ("fence", ops[i][1]) for o in ops[:i]) and any(o == ("fence", ops[i][1]) for o in ops[i:])
            if fenced:
                after[w, l, i].add((v, m, j))
    reach = {}

    def behind(n):
        seen, todo = set(), [n]
        while todo:
            for x in after[todo.pop()]:
                if x not in seen:
                    seen.add(x)
                    todo.append(x)
        return seen

    store, read = [i for i, o in enumerate(ops) if o[0] == "store"][0], len(ops) - 1
    for lane in range(LANES):
        reach[lane] = behind(("a", lane, store))
    return [(l, m) for l in range(LANES) for m in range(LANES) if ("b", m, read) not in reach[l]]


def test_every_read_comes_after_every_store():
    ops = kernel_operations()
    assert ops[0][0] == "store" and ops[-1][0] == "read" and sum(o[0] == "count" for o in ops) == 1
    assert unordered(ops) == []


RIGHT = [("store", False), ("barrier", False), ("fence", True), ("count", True), ("fence", True), ("barrier", False),
         ("shuffle", False), ("read", False)]


@pytest.mark.parametrize("gone", [1, 2, 4, 5])
def test_each_of_its_steps_is_needed(gone):
    assert unordered(RIGHT) == []
    assert unordered(RIGHT[:gone] + RIGHT[gone + 1:]) != []
