"""Sizes of dense 8-bit products with the tile that the library chooses for them on 256 compute
units: (fast, tile rows, tile columns, rows, inner, cols)."""

# more tiles than workgroups, rows that end one past a block of 16
WALKS = [
    (True, 256, 256, 4353, 400, 5400), (True, 128, 256, 2305, 400, 6456),
    (True, 256, 128, 6561, 400, 2312), (True, 128, 128, 1537, 400, 4944),
    (False, 160, 256, 2561, 400, 5904), (False, 256, 128, 6161, 400, 1800),
    (False, 128, 128, 4097, 528, 2832), (False, 64, 256, 5841, 400, 1544),
]
# the same with columns that are no multiple of eight
ODD_WALKS = [
    (True, 256, 256, 6545, 1936, 3727), (True, 128, 256, 2561, 400, 5931),
    (True, 256, 128, 2177, 400, 5379), (True, 128, 128, 4881, 400, 1547),
    (False, 160, 256, 2817, 400, 5389), (False, 256, 128, 2177, 400, 5415),
    (False, 128, 128, 1281, 400, 5661), (False, 64, 256, 1441, 400, 5415),
]
# a tile to a workgroup, reductions of other lengths
SINGLE = [
    (True, 256, 256, 2906, 1168, 3864), (True, 128, 256, 1427, 1104, 3768),
    (True, 256, 128, 2692, 976, 2904), (True, 128, 128, 774, 704, 1032),
    (False, 160, 256, 2718, 1472, 3464), (False, 256, 128, 1106, 336, 3784),
    (False, 128, 128, 2691, 560, 1360), (False, 64, 256, 707, 1136, 2848),
]
# reductions split over workgroups (the large tiles of fast are not split at these sizes)
SPLIT = [
    (True, 128, 256, 129, 7440, 5400), (True, 128, 128, 811, 3296, 536),
    (False, 160, 256, 130, 6992, 5424), (False, 256, 128, 197, 7824, 2696),
    (False, 128, 128, 1412, 3600, 624), (False, 64, 256, 851, 4464, 2168),
]
