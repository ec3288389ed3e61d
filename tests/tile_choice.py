"""Which tile the integer and the grouped products take, by their own cost models: the constants
are read from the sources, the formulas are written here again, so that a test can say which
kernel its shape is meant for."""
import math
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "microscaling_fp4_quantization_amd", "csrc")
CUS = 256
RANGES = [1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64]


def costs(name):
    text = open(os.path.join(CSRC, name)).read()
    table = re.search(r"constexpr TileCost kTileCosts\[\] = \{(.*)\};", text).group(1)
    return [tuple(float(v) for v in row.split(",")) for row in re.findall(r"\{([^{}]*)\}", table)]


def up(n, m):
    return -(-n // m)


def int8(m, n, k):
    """(tile, K ranges, quarter tiles) of int8_gemm; tile 0: at most 16 rows."""
    if m <= 16:
        return 0, 1, 0
    blocks, best, least = up(k, 128), (128, 1, 0), 1e300
    for tile, per_cu, alone, each, fixed in costs("fp4q_int8.hip"):
        tile, per_cu = int(tile), int(per_cu)
        tiles = up(m, tile) * up(n, tile)
        for sp in RANGES:
            per = up(blocks, sp)
            if sp > 1 and (sp > blocks or tiles * sp > 4 * CUS or 4 * sp * m * n > 1 << 28):
                break
            if sp > 1 and per * (sp - 1) >= blocks:
                continue
            quarters = tiles % CUS if tile == 256 and sp == 1 and tiles > CUS and tiles % CUS <= CUS // 4 else 0
            groups = up(tiles * sp - quarters, CUS)
            full, rest = divmod(groups, per_cu)
            t = full * (per * max(alone, each * per_cu) + fixed)
            if rest:
                t += per * max(alone, each * rest) + fixed
            if quarters:
                t += per * 0.6 + 4.0
            if sp > 1:
                t += 4.0 + 8.0 * sp * m * n / 8e6
            if t < least:
                least, best = t, (tile, sp, quarters)
    return best


def _grouped(wide, blocks, tiles):
    best, least = 128, 1e300
    for tile, per_cu, alone, each, each_wide, fixed in costs("fp4q_grouped.hip"):
        if wide and each_wide == 0.0:
            continue
        cost, groups = each_wide if wide else each, tiles(int(tile)) / CUS
        full = math.floor(groups / per_cu)
        rest = groups - full * per_cu
        t = full * (blocks * max(alone, cost * per_cu) + fixed)
        if rest > 0:
            t += blocks * max(alone, cost * rest) + fixed
        if t < least:
            least, best = t, int(tile)
    return best


def grouped(rows, groups, n, k, f32):
    """Tile of the grouped product over `groups` groups (of the linear layer: and the rows of none); 0: a pass over the weights."""
    some = min(rows, groups)
    if rows <= 8 * some:
        return 0
    return _grouped(f32, up(k, 128), lambda t: max(some, rows / t + 0.5 * some) * up(n, t))


def outer(rows, experts, m, n, f32):
    """Tile of the weight gradient, m x n per expert."""
    return _grouped(f32, rows / 128 / experts + 0.5, lambda t: experts * up(m, t) * up(n, t))
