"""How a thread block of the gated scan hands tiles from the warp that draws
tickets to those that compute, with few lanes: every interleaving of a model of
its named barriers (no GPU needed). The tile to bring to L2 is read between two
barriers that its writer only arrives at, so its slots must take turns."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "selective_state_space_12_b200", "csrc", "gated.cu")
WARPS, ROUNDS = 2, 3  # warps that compute, tiles


def programs(slots):
    chain, compute = [], []
    for n in range(ROUNDS):
        chain += [("arrive", "maps"), ("wait", "maps"), ("arrive", "entry"),
                  ("write", (n + 1) % slots), ("written", (n + 1) % slots), ("arrive", "ticket")]
        compute += [("arrive", "maps"), ("read", n % slots), ("done", n % slots),
                    ("arrive", "entry"), ("wait", "entry"), ("arrive", "ticket"),
                    ("wait", "ticket")]
    return [chain] + [compute] * WARPS


def overlaps(slots):
    """Whether some interleaving reads a slot while it is being written."""
    progs = programs(slots)
    seen, stack, ended = set(), [(0,) * len(progs)], False
    while stack:
        at = stack.pop()
        if at in seen:
            continue
        seen.add(at)
        past = [p[:k] for p, k in zip(progs, at)]
        arrived = {b: sum(s.count(("arrive", b)) for s in past) for b in ("maps", "entry", "ticket")}
        writing = {s[-1][1] for s in past[:1] if s and s[-1][0] == "write"}
        reading = {s[-1][1] for s in past[1:] if s and s[-1][0] == "read"}
        if writing & reading:
            return True
        ended = ended or all(k == len(p) for p, k in zip(progs, at))
        for w, (p, k) in enumerate(zip(progs, at)):
            if k < len(p):
                kind, what = p[k]
                phase = past[w].count(("arrive", what))
                if kind != "wait" or arrived[what] >= phase * len(progs):
                    stack.append(at[:w] + (k + 1,) + at[w + 1:])
    assert ended, "the model's barriers do not end"
    return False


def test_the_model_sees_one_slot_overlap():
    assert overlaps(1) and not overlaps(2)


def test_the_tile_to_fetch_ahead_has_slots_enough():
    with open(SOURCE, encoding="utf-8") as f:
        src = f.read()
    slots = re.search(r"\bTile later(?:\[(\d+)\])?;", src)
    assert not overlaps(int(slots.group(1) or 1))
    uses = set(re.findall(r"\bs\.later(\[[^\]]*\])?", src))
    assert uses == {"[0]", "[n & 1]", "[(n + 1) & 1]"}, uses
