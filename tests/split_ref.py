"""How fa_split.cuh cuts a ragged batch, restated in Python for the tests: the plan from the sizes, each
unit's first piece and number of pieces from the lengths, and the pieces that the joining kernel reads."""


def ceil(a, b):
    return -(-a // b)


class Plan:
    def __init__(self, B, per_seq, slots, least, share, most_tiles):
        """most_tiles: key tiles of the longest sequence that the tensors can hold."""
        units = B * per_seq
        few = 2 * units <= slots
        self.B, self.per_seq, self.units, self.slots, self.least = B, per_seq, units, slots, least
        self.items = units if B > 512 or most_tiles <= least else slots if few else units + (4 * slots + share - 1) // share
        self.share = 0 if few else share
        self.room = 2 * (self.items - units)  # pieces that the workspace holds


def cross_plan(B, Hq, Hkv, Tq, Tk, sms):
    """Of the few-rows kernel of cross attention: (plan, rows of a unit)."""
    rows = Hq // Hkv * Tq
    return Plan(B, Hkv * ceil(rows, 128), 2 * sms, 1, 7, ceil(Tk, 128)), min(rows, 128)


def tree_plan(B, Hq, Hkv, N, slots, sms):
    rows = Hq // Hkv * N
    return Plan(B, Hkv * ceil(rows, 128), sms, 3, 4, slots / 128), min(rows, 128)


def units_of(p, tiles):
    """{unit: (part, pieces)} for the sequences' key tiles."""
    if p.items == p.units:
        return {u: (0, 1) for u in range(p.units)}

    def pieces(t, c):
        return max(1, ceil(t, c))

    least, total = max(1, p.least), sum(tiles)
    if p.B <= 128:
        lo, hi = least, max(least, max(tiles))
        while lo < hi:
            c = (lo + hi) // 2
            if sum(pieces(t, c) for t in tiles) * p.per_seq <= p.items:
                hi = c
            else:
                lo = c + 1
        chunk = lo
    else:
        chunk = max(least, ceil(total * p.per_seq, p.items - p.units))
    if p.share:
        chunk = max(chunk, total * p.per_seq * p.share // (4 * p.slots))
    order = range(p.B)
    if p.B <= 32:  # longer pieces first
        order = sorted(order, key=lambda b: (-(tiles[b] // pieces(tiles[b], chunk)), b))
    out, number, rank = {}, 0, 0
    for b in order:
        n = pieces(tiles[b], chunk)
        for unit in range(p.per_seq):
            out[b * p.per_seq + unit] = (2 * (number - rank), n)
            number += n
            rank += 1
    assert number <= p.items
    return out


def joined(units):
    """The pieces that the joining kernel reads: units of one piece have been finished by their CTA."""
    return [range(part, part + pieces) for part, pieces in units.values() if pieces > 1]
