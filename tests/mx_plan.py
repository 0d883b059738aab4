"""Which kernel a product on MX FP4 lines takes, for tests that have to reach each of them: the
rule of mxfp4_linear.hip written again (tests/test_feedforward_abi_cpu.py holds it against the
library's workspace query), and sizes that take every kernel through its steady state."""

CODE_STAGES = {"small": 5, "mid": 4, "large": 2}    # steps of codes in a tile's ring
SCALE_BUFFERS = {"small": 3, "mid": 2, "large": 2}  # groups of four steps of scales


def steps_of(k):
    return -(-k // 256)


def plan(m, n, k, gated):
    """(kernel, splits of K): a tile's name, or ("stream", rows of X it has room for, columns of C
    in sixteens)."""
    steps, wide = steps_of(k), 2 * n if gated else n
    if m <= 64:
        cols = 32 if -(-n // 16) > (512 if m <= 8 and not gated else 256) else 16
        rows = next(r for r in (8, 16, 32, 64) if m <= r)
        splits = min(256 // -(-n // cols), steps // 32)
        return ("stream", rows, cols // 16), max(splits, 1)
    best = None
    for shape, bm, bn, fixed, step in (("small", 64, 128, 5.0, 0.53), ("mid", 128, 128, 7.2, 0.71),
                                       ("large", 256, 256, 9.5, 1.75)):
        tiles = -(-m // bm) * -(-wide // bn)
        for splits in range(1, 17):
            if splits > 1 and (tiles * splits > 256 or steps // splits < 4):
                break
            time = -(-tiles * splits // 256) * (fixed + step * -(-steps // splits))
            if splits > 1:
                time += 4.0 + splits * m * wide * 4.0 / 3.5e6
            if best is None or time < best[0]:
                best = (time, shape, splits)
    return best[1], best[2]


# Tiles: from one ring's steps to many times around it, odd and even, ragged everywhere, and with
# rows of 16-bit outputs at multiples of 16 bytes; K whole, then split, with odd first steps among
# the splits.
TILES = ([(m, n, 256 * steps - 57) for m, n in ((2900, 4501), (1500, 1300), (1025, 1030))
          for steps in (5, 8, 9, 13, 17, 33)]
         + [(2900, 300, 6343), (65, 4500, 6343)]
         + [(2900, 4504, 2247), (1500, 1304, 2247), (1025, 1032, 2247)]
         + [(513, 4500, 18119), (2050, 130, 32455), (130, 3001, 19143), (130, 4500, 32455),
            (65, 4500, 12999), (130, 2050, 12999), (2050, 2050, 17000), (1001, 513, 30001),
            (100, 75, 60001)])

# Few rows: 16 and 32 columns a workgroup at each number of rows, one step, steps that are not
# shared evenly by eight waves, and more than a wave's ring holds; K split in the last ones.
STREAM = ([(m, n, k) for m in (1, 8, 12, 16, 24, 32, 37, 64) for n in (700, 4113, 8209)
           for k in (200, 3271, 8391)]
          + [(m, 70, 70001) for m in (1, 8, 12, 16, 24, 32, 37, 64)])
