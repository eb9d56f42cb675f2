"""The order that the barriers of cross attention's forward give its ring of key and value tiles (csrc/lm_attn_fwd.cuh), as a
model: the loader fills slots in turn (K_0, V_0, K_1, ...), a warp looks at every fill and clears what nobody sees, the tensor
cores take a K when it is full and a V when it is clear, and a slot is filled again when its products are done and that
warp has been there.  Waits ask for a phase's parity, as the hardware does.  Every order of the steps is walked: none ends
with all waiting, and no wait is passed by another phase than its own."""
import pytest


def _walk(slots, tiles, both):
    """(states, what is wrong); both: a free slot waits for the clearing warp too, not for the products alone."""
    fills, arrivals = 2 * tiles, 2 if both else 1
    products = [("k", 0)]
    for i in range(tiles):
        products += [("k", i + 1)] * (i + 1 < tiles) + [("v", i)]
    zero = (0,) * slots
    start = (0, 0, 0, zero, zero, zero, frozenset())
    seen, left, wrong = {start}, [start], set()

    def up(t, i):
        return t[:i] + (t[i] + 1,) + t[i + 1:]

    def passes(done, phase):  # try_wait.parity: some phase of this parity is over, and none of the other since
        return (done & 1) != (phase & 1)

    while left:
        asked, made, looked, full, empty, clean, flying = left.pop()
        after = []
        if asked < fills:
            s, f = asked % slots, asked // slots
            if passes(empty[s] // arrivals, f - 1):
                if empty[s] // arrivals != f:
                    wrong.add("a slot filled too early")
                after.append((asked + 1, made, looked, full, empty, clean, flying | {asked}))
        for n in flying:
            after.append((asked, made, looked, up(full, n % slots), empty, clean, flying - {n}))
        if made < len(products):
            kind, i = products[made]
            n = 2 * i + (kind == "v")
            s, f, there = n % slots, n // slots, clean if kind == "v" else full
            if passes(there[s], f):
                if there[s] != f + 1:
                    wrong.add("a product of another tile")
                after.append((asked, made + 1, looked, full, up(empty, s), clean, flying))
        if looked < fills:
            s, f = looked % slots, looked // slots
            if passes(full[s], f):
                if full[s] != f + 1:
                    wrong.add("another tile cleared")
                after.append((asked, made, looked + 1, full, up(empty, s) if both else empty, up(clean, s), flying))
        if not after and (asked, made, looked) != (fills, len(products), fills):
            wrong.add("all wait")
        for state in after:
            if state not in seen:
                seen.add(state)
                left.append(state)
    return len(seen), wrong


@pytest.mark.parametrize("slots", [5, 8])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 7, 11])
def test_no_order_of_the_steps_stops(slots, tiles):
    states, wrong = _walk(slots, tiles, True)
    assert states > tiles and not wrong


def test_a_slot_that_waits_for_its_products_alone_is_not_enough():
    assert _walk(5, 3, False)[1] == {"all wait"}
