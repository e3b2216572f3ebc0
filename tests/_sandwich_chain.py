"""How many roundings stand between a term and its sum in the sandwich norms' kernels, counted from how
they share the work.  u = 2^-24, what one fp32 rounding is off by at most, relative to its result.

A row's sum of squares: a thread has up to four 16-byte vectors, 32 values, as four partial sums of up
to eight fused multiply-adds; two additions join those, five the lanes of a warp, and the warps' parts
(a multiple of four places for each CTA, up to 24 in all) take up to seven: 22 u.  The mean adds 2 u,
the root halves that, its Newton step adds 2 u: a statistic is within 14 u.  A stored value has five
more roundings before its own (the row vectors' product 2, its two products and the sum): under 32 u
of the magnitudes of its terms.

The backward pass takes the statistics as given.  A row's sum: up to 16 fused multiply-adds in a
thread, one to join its halves, five in a warp, up to five for the warps, and 4 u in a term: 31 u; with
the mean and its factor 34 u; so dh, which is a term (4 u) and that times hh, is within 38 u of its
terms, and dh * uh within 40: under 48 u.  grad_update has a mean of two such sums' difference, one
times the mean of the other: under 128 u."""

VALUE, TERM, UPDATE = 32, 48, 128  # a stored value, a term of a column's sum, grad_update


def shape(Dv, backward):
    """-> (vectors of a CTA's part of a row, a thread's vectors, warps of a group, groups)."""
    nv = (Dv + 1) // 2 if Dv > 1024 else Dv

    def with_(v):
        warps = -(-nv // (32 * v))
        return nv, v, warps, (8 if backward and v > 2 else 16) // warps

    if nv <= 64:
        return with_(1 if nv <= 32 else 2)
    used = {v: with_(v)[3] * nv * 12 // v for v in (3, 4)}
    return with_(3 if used[3] > used[4] else 4)


def items(S, D):
    """Of the backward pass: -> (rows of an item, items of a batch, groups at work)."""
    groups = shape(D // 8, True)[3]
    over = 76 if D > 8192 else 152
    rounds = -(-S // (256 * over))
    rows = max(-(-S // (rounds * over)), 2 * groups if groups > 4 else 8)
    rows = min(rows, S)
    return rows, -(-S // rows), min(rows, groups)


def column_additions(B, S, D, shared):
    """Additions that a term of a column's sum goes through, beside its own roundings: the rows of a
    group, its CTA's groups in pairs, the items in `ks` slices, the slices, and where the sum is over
    the batches too, those that a warp takes and the warps."""
    rows, n, groups = items(S, D)
    ks = 4
    while ks < 32 and ks < n:
        ks *= 2
    count = -(-rows // groups) + (groups - 1).bit_length() + -(-n // ks) + ks
    if shared:
        at_once = 64 // ks
        count += -(-B // at_once) + min(B, at_once)
    return count
