"""The hand-off of key halves in k_weights_tiles, walked through exhaustively on
the host: the copies, the key warps (two stand for eight) and the products, with
the barriers' counts and parities as the kernel has them.  A product must find a
half written by every key warp."""
import os
import re

import pytest

RAW, HALVES, WARPS = 3, 3, 2
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "compressed_sparse_attention_layer_gb300", "csrc", "csa2_attn_weights.cu")


class Bar:
    """(arrivals in the running phase, phases completed) of an mbarrier that expects `count`."""

    @staticmethod
    def arrive(bar, count):
        return (0, bar[1] + 1) if bar[0] + 1 == count else (bar[0] + 1, bar[1])

    @staticmethod
    def done(bar, phase):                          # what a test of phase's parity says
        return (bar[1] & 1) != (phase & 1)


def put(t, i, v):
    return t[:i] + (v,) + t[i + 1:]


def faults(tiles, stop_waits):
    """What some schedule leads to: "early", a product reads a half that a key warp has yet to write; "stuck",
    a wait that nothing ends."""
    # A key warp's steps: tile p: 0 wait full and leave the page, 1 and 2 the halves; then the stop.
    zero = ((0, 0),)
    # copies: tile; warps: (tile, step); product: (tile, half); barriers; written[slot]: per warp the half it holds
    start = (0, ((0, 0),) * WARPS, (0, 0), zero * RAW, zero * RAW, zero * HALVES, zero * HALVES,
             ((None,) * WARPS,) * HALVES)
    seen, todo, found = {start}, [start], set()
    while todo:
        cp, warps, prod, full, empty, kready, kfree, written = todo.pop()
        nxt = []
        if cp <= tiles:                            # the page (or the stop) of product cp
            i = cp % RAW
            if cp < RAW or Bar.done(empty[i], cp // RAW - 1):
                nxt.append((cp + 1, warps, prod, put(full, i, Bar.arrive(full[i], 1)), empty, kready, kfree, written))
        for w, (p, step) in enumerate(warps):
            if p > tiles:
                continue
            i, half = p % RAW, 2 * p + max(step - 1, 0)
            slot, turn = half % HALVES, half // HALVES
            if step == 0:
                if not Bar.done(full[i], p // RAW):
                    continue
                if p < tiles:
                    nxt.append((cp, put(warps, w, (p, 1)), prod, full, put(empty, i, Bar.arrive(empty[i], WARPS)),
                                kready, kfree, written))
                elif not stop_waits or turn == 0 or Bar.done(kfree[slot], turn - 1):
                    nxt.append((cp, put(warps, w, (p + 1, 0)), prod, full, empty,
                                put(kready, slot, Bar.arrive(kready[slot], WARPS)), kfree, written))
            elif turn == 0 or Bar.done(kfree[slot], turn - 1):
                nxt.append((cp, put(warps, w, (p, 2) if step == 1 else (p + 1, 0)), prod, full, empty,
                            put(kready, slot, Bar.arrive(kready[slot], WARPS)), kfree,
                            put(written, slot, put(written[slot], w, half))))
        p, h = prod
        if p <= tiles:
            half = 2 * p + h
            slot, turn = half % HALVES, half // HALVES
            if Bar.done(kready[slot], turn):
                if p < tiles:
                    if any(x != half for x in written[slot]):
                        found.add("early")
                    nxt.append((cp, warps, (p, 1) if h == 0 else (p + 1, 0), full, empty, kready,
                                put(kfree, slot, Bar.arrive(kfree[slot], 1)), written))
                else:
                    nxt.append((cp, warps, (p + 1, 0), full, empty, kready, kfree, written))
        if not nxt and not (cp == tiles + 1 and prod == (tiles + 1, 0) and all(p == tiles + 1 for p, _ in warps)):
            found.add("stuck")
        for s in nxt:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return found


@pytest.mark.parametrize("tiles", range(0, 9))
def test_no_product_reads_a_half_that_a_warp_has_yet_to_write(tiles):
    assert faults(tiles, stop_waits=True) == set()


def test_the_walk_sees_a_stop_that_does_not_wait():
    assert ["early" in faults(t, stop_waits=False) for t in range(5)] == [False, False, True, True, True]


def test_the_kernels_stop_waits_for_its_place():
    """The arrival of a key warp at the stop follows a wait for the half's place, as every other does."""
    src = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    src = src[src.index("k_weights_tiles"):src.index("AM_KEYS")]
    stops = re.findall(r"if \(m\.flags & AP_STOP\) \{(.*?mbar_arrive\(&S\.kready\[slot\]\).*?)\n            \}", src, re.S)
    assert len(stops) == 1
    wait, arrive = stops[0].find("&S.kfree[slot], turn - 1"), stops[0].find("mbar_arrive(&S.kready[slot])")
    assert 0 <= wait < arrive
