"""When the grouped chunk attention shares an item's keys out over thread blocks (no GPU needed)."""


def test_wide_heads_have_half_the_places(lib):
    """Two thread blocks an SM up to 128 channels, one of 256: 304 and 152 places.  In tables of 2048 tokens, too
    short for a smaller last part, items are shared out where two parts of each find places."""
    needed = lib.paged_attn_chunk_workspace_needed
    for items in range(1, 400):
        for dim, most in ((64, 152), (128, 152), (256, 76)):
            assert (needed(items, 4, 1, dim, 16, 128, 1) > 0) == (items <= most), (items, dim)
            assert (needed(1, 4 * items, items, dim, 16, 128, 1) > 0) == (items <= most), (items, dim)


def test_a_smaller_last_part_takes_the_places_left_over(lib):
    """In long tables, as far as nine items share one such place."""
    needed = lib.paged_attn_chunk_workspace_needed
    for items in range(1, 400):
        for dim, places in ((64, 304), (128, 304), (256, 152)):
            left = places - items
            pays = items <= places // 2 or (left > 0 and -(-items // left) <= 9)
            assert (needed(items, 4, 1, dim, 16, 4096, 1) > 0) == pays, (items, dim)


def test_the_workspace_is_as_large_as_ever(lib):
    for dim in (64, 128, 256):
        assert lib.paged_attn_chunk_workspace_size(1, 4, 1, dim, 16, 4096, 1) == 608 * 128 * (dim + 2) * 4
