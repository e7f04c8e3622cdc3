"""Products whose units take several output tiles over rows that stay (T, E, topk, cols, outs,
block_m), and what their plans at 152 SMs have to show: outputs of a tile, windows of blocks, parts of
a block, a last unit with fewer tiles, a last tile with fewer outputs."""

STAYING = [
    # shape,                        tile, windows, parts, short unit, short tile
    ((500, 300, 2, 384, 1432, 128), 192, False, False, False, True),
    ((500, 300, 2, 512, 2000, 128), 192, False, False, True, True),
    ((6000, 896, 8, 288, 1432, 128), 192, False, False, False, True),   # every tile in one unit
    ((500, 300, 4, 384, 1536, 256), 192, False, True, False, False),
    ((500, 300, 2, 384, 1432, 256), 192, False, True, True, True),
    ((500, 300, 2, 512, 1432, 8), 192, True, False, False, True),
    ((500, 300, 2, 64, 2000, 8), 192, True, False, True, True),
    ((9000, 300, 4, 64, 640, 128), 128, False, False, True, False),
    ((500, 300, 2, 512, 640, 256), 128, False, True, True, False),
    ((9000, 300, 4, 512, 640, 8), 128, True, False, True, False),
    ((96, 220, 5, 576, 1400, 1), 128, True, False, True, True),
    ((14, 434, 15, 544, 272, 512), 96, False, True, True, True),
    ((772, 462, 3, 32, 648, 1), 96, True, False, True, True),
    ((56, 512, 13, 352, 408, 1), 96, True, False, True, True),
    ((175, 960, 7, 544, 280, 1), 96, True, False, True, True),
]


def plan_row(plan, outs):
    return (plan.tile_outs, plan.window > 1, plan.parts > 1, plan.tiles % plan.unit_tiles != 0,
            outs % plan.tile_outs != 0)
