"""Which kernel a product with 4-bit weights takes, by the library's rule in plain Python, and
products that bring each of them past its first steps."""

CUS = 256
WAVES = dict(narrow=8, middle=8, stream=4)     # of a streamed kernel's workgroup, along the row


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


def slabs_of_waves(kernel, row_len):
    """Slabs of 128 inputs of each wave of a streamed kernel, the last one's part slab among them."""
    slabs = -(-row_len // 128)
    per = -(-slabs // WAVES[kernel])
    return [min(slabs, (w + 1) * per) - min(slabs, w * per) for w in range(WAVES[kernel])]


# (tokens, rows, experts, outputs, row length): three slabs and more for a wave, odd and even numbers of
# them, with a last slab that the rows end in
LONG = {
    "narrow": [(8, 8, 8, 250, 3300), (30, 45, 2, 70, 2350)],
    "middle": [(8, 8, 8, 1024, 3300), (20, 60, 3, 1050, 2350)],
    "stream": [(200, 200, 3, 1100, 2050), (90, 250, 5, 900, 1900)],
}
STREAMED = [(*shape, group) for shapes in LONG.values() for shape in shapes for group in (32, 64, 128)]
STREAMED += [(8, 8, 8, 1024, 3300, 384), (200, 200, 3, 1100, 2050, 256)]

# rows whose last slab holds fewer groups than a full one, in each kernel
PART_SLABS = [(9, 40, 3, 33, 300, 32), (9, 40, 3, 33, 150, 64), (20, 60, 3, 1050, 400, 32), (20, 60, 3, 1050, 420, 64),
              (200, 200, 3, 1100, 340, 32), (200, 200, 3, 1100, 300, 64), (300, 1200, 8, 1500, 130, 32),
              (400, 1600, 8, 1400, 190, 64), (300, 1200, 8, 2500, 300, 32), (200, 1300, 8, 2400, 180, 64)]
