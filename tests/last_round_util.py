"""What the offsets of a launch make of its last round, counted as the kernels do."""


def last_round(counts, N, rows, cols, steps, branches=1):
    """(parts of each tile of the last round, sums that they leave in scratch) of a product over groups of these rows
    with tiles of rows x cols of its N outputs at two blocks a CU: tiles in groups of eight row tiles over the columns,
    the last 512 or fewer of them in as many parts as fill 512 blocks, at most eight and of at least eight steps
    (of 128 bytes of the reduction) each; (1, 0) where they stay whole."""
    row_tiles = [min(rows, c - r) for c in counts for r in range(0, c, rows)]
    ptiles = -(-N // cols)
    n = len(row_tiles) * ptiles
    rest = n % 512
    parts = min(512 // rest, 8, steps // 8) if rest else 1
    if parts < 2:
        return 1, 0
    words = 0
    for t in range(n - rest, n):
        grp, rem = divmod(t, 8 * ptiles)
        cur = min(8, len(row_tiles) - grp * 8)
        words += row_tiles[grp * 8 + rem % cur] * min(cols, N - rem // cur * cols)
    return parts, words * parts * branches
