"""The compiled 256 x 256 product kernels, behind a tile: a workgroup that goes on to its next tile waits for that
tile's first stage by the number of operations issued since, among them the stores of the tile before.  Every round of
the loop over the tile's rows has to issue its share of them, and no load into LDS comes between them and that wait."""

from __future__ import annotations

import heapq
import re

from test_isa_linear256 import listing  # noqa: F401

STORES = 32             # that the waits count on
LOADS = 16              # of a stage, into LDS
ROUNDS = 4              # of the epilogue's loop over eight rows of blocks, two at a time
BEHIND = f"s_waitcnt vmcnt({LOADS + STORES}) lgkmcnt(0)"
FIRST = f"s_waitcnt vmcnt({LOADS}) lgkmcnt(0)"


def kernels(listing):  # noqa: F811
    for m in re.finditer(r"^(_ZN\S*kl_linear256ILi(\d)\S*):(.*?)^\.Lfunc_end", listing, re.S | re.M):
        yield m.group(1), int(m.group(2)), [x.split(";")[0].strip() for x in m.group(3).split("\n")]


def successors(lines):
    labels = {x[:-1]: i for i, x in enumerate(lines) if re.match(r"\.LBB\w+:$", x)}
    out = []
    for i, x in enumerate(lines):
        b = re.match(r"s_(c?)branch\S*\s+(\.LBB\w+)", x)
        assert not re.match(r"s_(setpc|swappc|cbranch_[ig]_fork)", x), x
        to = [] if x.startswith("s_endpgm") or (b and not b.group(1)) else [i + 1]
        if b:
            to.append(labels[b.group(2)])
        out.append([t for t in to if t < len(lines)])
    return out


def is_load(x):
    return x.startswith("buffer_load_dwordx4") and x.endswith("lds")


def is_store(x):
    return x.startswith("buffer_store_dwordx4")


def among_products(lines):
    """The loads into LDS of the main loop and a tile's last stages: products stand between one and the one before.  (Those
    that begin a workgroup's first tile stand together, and its wait is another one, chosen by a flag.)"""
    out, products = set(), False
    for i, x in enumerate(lines):
        products |= x.startswith("v_mfma")
        if is_load(x):
            if products:
                out.add(i)
            products = False
    return out


def epilogue_loops(lines, to):
    """The loops that hold stores and no products, as sets of lines: what is left of the cycles without the products."""
    keep = [not x.startswith("v_mfma") for x in lines]
    order, low, on, stack, found, count = {}, {}, set(), [], [], 0
    for root in range(len(lines)):
        if not keep[root] or root in order:
            continue
        work = [(root, iter(to[root]))]
        order[root] = low[root] = count
        count += 1
        stack.append(root)
        on.add(root)
        while work:
            i, it = work[-1]
            for t in it:
                if not keep[t]:
                    continue
                if t not in order:
                    order[t] = low[t] = count
                    count += 1
                    stack.append(t)
                    on.add(t)
                    work.append((t, iter(to[t])))
                    break
                if t in on:
                    low[i] = min(low[i], order[t])
            else:
                work.pop()
                if work:
                    low[work[-1][0]] = min(low[work[-1][0]], low[i])
                if low[i] == order[i]:
                    part = set()
                    while True:
                        j = stack.pop()
                        on.discard(j)
                        part.add(j)
                        if j == i:
                            break
                    if len(part) > 1 and any(is_store(lines[j]) for j in part):
                        found.append(part)
    return found


def fewest_stores(lines, to, loop, start):
    """Of a round of the loop, from `start` to `start`."""
    best, queue = {}, [(int(is_store(lines[start])), t) for t in to[start] if t in loop]
    while queue:
        d, i = heapq.heappop(queue)
        if i == start:
            return d
        if i in best:
            continue
        best[i] = d
        for t in to[i]:
            if t in loop:
                heapq.heappush(queue, (d + is_store(lines[i]), t))
    raise AssertionError("not a loop")


def test_every_round_behind_a_tile_stores_its_rows(listing):  # noqa: F811
    found = list(kernels(listing))
    assert len(found) == 6
    for name, mode, lines in found:
        assert lines.count(BEHIND) == 1 and lines.count(f"s_waitcnt vmcnt({STORES + 6})") == 1, name
        to = successors(lines)
        loops = epilogue_loops(lines, to)
        assert len(loops) == (1 if mode == 2 else 5), (name, len(loops))  # one an activation
        inside = set().union(*loops)
        edges = [(i, t) for i in range(len(lines)) for t in to[i]]
        into = [sorted({t for i, t in edges if t in loop and i not in loop}) for loop in loops]
        for loop, entries in zip(loops, into):
            assert len(entries) == 1, name
            # a weight gradient stores fp32, twice as much
            assert fewest_stores(lines, to, loop, entries[0]) * ROUNDS >= STORES * (2 if mode == 2 else 1), name
        assert all(i in inside for i, x in enumerate(lines) if is_store(x)), name


def test_no_load_into_lds_between_the_stores(listing):  # noqa: F811
    # (what begins a workgroup's first tile, whose wait is another one, is chosen by a flag that is never set here)
    for name, _, lines in kernels(listing):
        to, loads = successors(lines), among_products(lines)
        assert len(loads) >= 3 * LOADS - 1, name
        queue = [t for i, x in enumerate(lines) if is_store(x) for t in to[i]]
        seen = set()
        while queue:
            i = queue.pop()
            if i in seen or lines[i].startswith((BEHIND, FIRST, "v_mfma")):
                continue
            if is_load(lines[i]) and i not in loads:
                continue
            seen.add(i)
            assert i not in loads, (name, i, lines[i])
            queue += to[i]
