"""Shapes that reach every form of the orthogonalised update, for the GPU test
of the forms and the host test that nothing is left out."""

# (rows, cols, batch, products): rows and columns of a result tile (128 rows: one
# CTA, 256: a pair), which of the three products of a step split a tile's depth,
# units (CTAs or pairs) of a group more than one ("met") or not
FORMS = {
    # one CTA a tile
    (511, 385, 1, 1): (128, 128, (0, 0, 0), True),
    (1111, 259, 1, 1): (128, 128, (1, 0, 0), True),
    (600, 2300, 2, 1): (128, 128, (1, 0, 0), True),
    (300, 700, 90, 1): (128, 128, (0, 0, 0), True),      # two matrices to a group, in turn
    (40, 700, 3, 3): (128, 128, (1, 0, 0), True),
    (300, 700, 40, 3): (128, 128, (0, 0, 0), True),
    (2600, 130, 1, 3): (128, 128, (1, 0, 0), True),      # a second strip of row tiles, partly filled
    (590, 614, 1, 3): (128, 128, (1, 1, 0), True),
    (680, 662, 1, 3): (128, 128, (1, 1, 1), True),
    # pairs, 256 x 128
    (1356, 1096, 1, 1): (256, 128, (0, 0, 0), True),
    (4046, 1032, 1, 1): (256, 128, (1, 0, 0), True),
    (1110, 3251, 1, 1): (256, 128, (1, 0, 0), True),
    (2304, 2100, 2, 3): (256, 128, (0, 0, 0), True),     # several tiles to a pair, a second strip
    (669, 3650, 3, 3): (256, 128, (1, 0, 0), True),
    (1903, 700, 1, 3): (256, 128, (1, 0, 0), True),
    (1258, 1403, 1, 3): (256, 128, (1, 1, 0), True),
    # pairs, 256 x 256
    (768, 768, 12, 1): (256, 256, (0, 0, 0), True),      # nine tiles for six pairs, six symmetric blocks
    (2304, 2304, 1, 1): (256, 256, (0, 0, 0), True),     # 81 tiles for 76 pairs, a second strip
    (2500, 5200, 1, 1): (256, 256, (0, 0, 0), True),
    (5200, 2500, 1, 1): (256, 256, (0, 0, 0), True),
    (1004, 4540, 3, 1): (256, 256, (1, 0, 0), True),
    (331, 256, 63, 1): (256, 256, (0, 0, 0), False),
    (512, 819, 16, 3): (256, 256, (0, 0, 0), True),
    (232, 5649, 17, 3): (256, 256, (1, 0, 0), True),
    (4865, 137, 13, 3): (256, 256, (1, 0, 0), True),
    (160, 700, 200, 3): (256, 256, (0, 0, 0), False),    # a pair takes three matrices in turn
}

# Muon steps (three products): (rows, cols, batch)
MUON_FORMS = {
    (768, 2304, 1): (128, 128, (1, 1, 0), True),
    (2304, 1536, 2): (256, 128, (0, 0, 0), True),
    (1258, 1403, 1): (256, 128, (1, 1, 0), True),
    (669, 3650, 3): (256, 128, (1, 0, 0), True),
    (512, 819, 16): (256, 256, (0, 0, 0), True),
    (232, 5649, 17): (256, 256, (1, 0, 0), True),
    (133, 136, 51): (256, 256, (0, 0, 0), False),
}


def form_of(z, rows, cols, batch, products, muon=False, sms=152):
    """The form that a call takes, as above; None where each matrix stays in one SM."""
    p = z.zero_debug_matrix_plan(z.matrices(rows, cols, batch=batch, out_dtype=z.ZERO_BF16 if muon else z.ZERO_FP32,
                                            products=products), muon, sms)
    if p.tile_rows == 0:
        return p.products, None
    return p.products, (p.tile_rows, p.tile_cols, tuple(int(s > 1) for s in p.split), p.units > 1)
