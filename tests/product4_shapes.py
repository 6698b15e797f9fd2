"""Which kernel a product with 4-bit weights takes, by the library's rule in plain Python, and
products that bring each of them to its edges."""

CUS = 256


def kernel_of(rows, experts, outputs, row_len):
    """narrow, middle, stream (16 rows by 16, 32 or 64 outputs), square or wide (64 rows by 64 or
    128 outputs)."""
    parts = min(experts, rows)
    each = -(-rows // parts)

    def tiles(high, across):
        return parts * -(-each // high) * -(-outputs // across)

    large = tiles(64, 128)
    if row_len >= 128 and each >= 16 and large >= (CUS * 11 // 16 if each >= 64 else CUS):
        return "square" if large < CUS * 7 // 4 else "wide"
    n = tiles(16, 16)
    return "narrow" if n <= CUS else "middle" if n < 4 * CUS else "stream"


def groups_of_a_slab(group):
    return max(1, 128 // group)


# rows whose last slab holds fewer groups than a full one, in each kernel
PART_SLABS = [(9, 40, 3, 33, 300, 32), (9, 40, 3, 33, 150, 64), (20, 60, 3, 1050, 400, 32), (20, 60, 3, 1050, 420, 64),
              (200, 200, 3, 1100, 340, 32), (200, 200, 3, 1100, 300, 64), (300, 1200, 8, 1500, 130, 32),
              (400, 1600, 8, 1400, 190, 64), (300, 1200, 8, 2500, 300, 32), (200, 1300, 8, 2400, 180, 64)]
