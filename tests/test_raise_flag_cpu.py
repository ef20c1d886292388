"""The flag by which a group's warps agree to move their references (csrc/tree_attn_few.cu), as a model: every order in
which the warps' steps can happen.  A warp that finds the flag clear goes on to the next tile at once, so the next
tile's answer must not be written where a slower warp still looks for this one's."""
import itertools
import os

WARPS, TILES = 2, 3


def program(ups, flags):
    """One warp's steps.  Yields ("set" | "read" | "clear", tile's flag) or "barrier"; a read's answer is sent back."""
    for tile, up in enumerate(ups):
        at = tile % flags
        if up:
            yield ("set", at)
        yield "barrier"
        if (yield ("read", at)):
            yield "barrier"       # the warps' maxima are there
            yield ("clear", at)   # by one warp
            yield "barrier"       # the references have moved


def replay(ups, flags, warp, answers):
    """The warp's next step (None: it is through) after it was given `answers`, one for each step so far."""
    g = program(ups[warp], flags)
    try:
        step = next(g)
        for a in answers:
            step = g.send(a)
    except StopIteration:
        return None
    return step


def orders_agree(ups, flags):
    """Whether in every order all warps find each tile's flag set exactly if one of them set it, and none waits for good.
    The barrier is the kernel's: a count and a phase, of which a waiting warp sees the parity alone."""
    want = [any(u[t] for u in ups) for t in range(TILES)]
    start = (tuple((0,) * flags), 0, 0, tuple(((), 0, False) for _ in range(WARPS)))  # flags, arrived, phase, warps
    seen, todo = {start}, [start]
    while todo:
        flag, arrived, phase, warps = todo.pop()
        moved = done = 0
        for w, (answers, parity, waiting) in enumerate(warps):
            step = replay(ups, flags, w, answers)
            found = [a for a in answers if a is not None]
            if found != want[:len(found)]:
                return False
            if step is None:
                done += 1
                continue
            f, n, ph = list(flag), arrived, phase
            if waiting:
                if phase % 2 == parity:
                    continue
                nxt = (answers + (None,), parity ^ 1, False)
            elif step == "barrier":
                n += 1
                if n == WARPS:
                    n, ph = 0, ph + 1
                nxt = (answers, parity, True)
            elif step[0] == "read":
                nxt = (answers + (bool(f[step[1]]),), parity, False)
            else:
                if step[0] == "set" or w == 0:
                    f[step[1]] = int(step[0] == "set")
                nxt = (answers + (None,), parity, False)
            moved += 1
            new = (tuple(f), n, ph, warps[:w] + (nxt,) + warps[w + 1:])
            if new not in seen:
                seen.add(new)
                todo.append(new)
        if moved == 0 and done < WARPS:
            return False
    return True


EVERY = [list(zip(*[iter(bits)] * TILES)) for bits in itertools.product((False, True), repeat=WARPS * TILES)]


def test_two_flags_by_tile_parity_agree_in_every_order():
    assert all(orders_agree(ups, 2) for ups in EVERY)


def test_the_model_finds_the_race_of_a_single_flag():
    assert not all(orders_agree(ups, 1) for ups in EVERY)


def test_the_kernel_has_a_flag_for_either_parity():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "hierarchical_sparse_attention_block_b200", "csrc", "tree_attn_few.cu")) as f:
        source = f.read()
    assert "raise_flags + 2 * t + buf" in source and "buf = cnt & 1" in source
