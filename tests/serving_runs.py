"""The division of s2attn_tree_decode restated: how many runs a unit's key tiles are cut into, and which
tiles of which sequence a run takes.  A unit is a key head and a tile of up to 128 query rows."""

SEQ_COST = 3       # what a sequence's end weighs, in key tiles
SLOTS = 2 * 148    # CTAs of one wave


def plan(M, H, Hkv):
    """(tokens of a row tile, row tiles, runs J, rows of a partial)."""
    group = H // Hkv
    tok = 128 // group
    row_tiles = -(-M // tok)
    units = Hkv * row_tiles
    best, runs, J = None, 1, 1
    while J == 1 or units * J <= 2 * SLOTS:
        waves = -(-units * J // SLOTS)
        cost = (1.0 if units * J <= SLOTS else 1.2 * waves) / J
        if best is None or cost < best - 1e-9:
            best, runs = cost, J
        J += 1
    return tok, row_tiles, runs, min(tok, M) * group


def tiles_of(lens, new, first_tok):
    return [-(-n // 64) + -(-m // 64) if m > first_tok else 0 for n, m in zip(lens, new)]


def segments(lens, new, first_tok, J):
    """[(run, sequence, first tile, tiles, tiles of the sequence)] and the tiles of each sequence."""
    tiles = tiles_of(lens, new, first_tok)
    weight = sum(t + SEQ_COST for t in tiles if t)
    runs = min(J, max(1, sum(tiles)))
    each, more = divmod(weight, runs)

    def cut(w):
        """(sequence, tile) where weight w falls; behind a sequence's tiles: the next one's start."""
        before = 0
        for b, t in enumerate(tiles):
            if not t:
                continue
            if before + t + SEQ_COST > w:
                at = min(t, w - before)
                return (b, at) if at < t else (b + 1, 0)
            before += t + SEQ_COST
        return len(tiles), 0
    out = []
    for j in range(runs):
        w0 = each * j + min(j, more)
        (b0, t0), (b1, t1) = cut(w0), cut(w0 + each + (j < more))
        for b in range(b0, min(b1 + 1, len(tiles))):
            lo, hi = (t0 if b == b0 else 0), (t1 if b == b1 else tiles[b])
            if lo < hi:
                out.append((j, b, lo, hi - lo, tiles[b]))
    return out, tiles
