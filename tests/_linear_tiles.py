"""Shapes of the linear layers by the tiles that they are to take: every form, whole and cut along the
reduction, with few experts and with a tile table, ragged rows in both bands of a tile."""
from __future__ import annotations

import routing_expert_ffn_router_amd as moe

CUS, SCAN = 256, 64  # CUs; the most experts without a tile table
FIRST, SLACK = 2, 3  # rows before and behind the experts'


def ragged(E, seed, most, total=None):
    """Row counts of E experts: some none, some few, up to `most`; the last takes what `total` leaves."""
    counts = []
    for e in range(E):
        v = (e * 2654435761 + seed * 40503) % 65536
        counts.append(0 if v % 5 == 0 else 1 + v % 17 if v % 5 == 1 else 1 + v * most // 65536)
    if total is not None:
        while sum(counts) > total:
            counts[counts.index(max(counts))] //= 2
        counts[-1] += total - sum(counts)
    return counts


# (dtype, rows and columns of a tile, cut, counts, K, N)
CASES = [
    ("bf16", 64, 256, False, [0, 37, 17, 64, 1, 33, 0, 20], 1024, 2176),
    ("bf16", 64, 256, True, [0, 37, 17, 50, 1, 0, 16, 7], 2048, 2176),
    ("bf16", 64, 256, True, [65, 0, 3], 4096, 5504),
    ("bf16", 64, 256, False, ragged(70, 1, 60), 640, 384),
    ("bf16", 64, 256, True, ragged(70, 2, 45), 2048, 256),
    ("bf16", 128, 256, False, [130, 0, 77, 250], 1024, 2176),
    ("bf16", 128, 256, True, [130, 0, 77, 250], 2048, 2176),
    ("bf16", 128, 256, True, [0, 128, 300, 31, 5, 64, 0, 130], 6144, 8192),
    ("bf16", 128, 256, False, ragged(70, 3, 200, 8000), 384, 384),
    ("bf16", 128, 256, True, ragged(70, 3, 200, 8000), 6144, 128),
    ("bf16", 256, 256, False, [900, 0, 601], 1024, 896),
    ("bf16", 256, 256, True, [900, 0, 601], 2048, 896),
    ("bf16", 256, 256, True, [257, 700, 0, 33, 1000, 511, 2, 1300], 6144, 4096),
    ("bf16", 256, 256, False, ragged(66, 4, 300, 9000), 256, 384),
    ("bf16", 256, 256, True, ragged(66, 4, 300, 9000), 6144, 128),
    ("f32", 128, 256, False, [1200, 0, 333, 64, 900, 17, 1, 1500], 512, 4224),
    ("f32", 128, 256, True, [1200, 0, 333, 64, 900, 17, 1, 1500], 3200, 4096),
    ("f32", 128, 256, True, [4600], 4096, 4096),
    ("f32", 128, 256, False, ragged(70, 5, 200, 8000), 256, 2048),
    ("f32", 128, 256, True, ragged(66, 6, 200, 8000), 3200, 1920),
    ("bf16", 64, 32, False, [0, 37, 17, 64, 1, 33], 1024, 640),
    ("f32", 64, 64, False, [0, 137, 17, 64, 1, 33], 1024, 640),
    # a shape that may be cut, and rows whose last round is too full for it
    ("bf16", 256, 256, False, [1024, 1024, 1024, 1024], 6144, 4096),
]


def shape_of(case):
    dtype, _, _, _, counts, K, N = case
    return moe.group_shape(FIRST + sum(counts) + SLACK, len(counts), N, K,
                           moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32)


def pieces_of(case):
    """Pieces that the last round's tiles are cut into, from the rows there are."""
    rows, columns, most = moe.linear_tiles(shape_of(case))
    tiles = sum(-(-n // rows) for n in case[4]) * -(-case[6] // columns)
    tail = tiles % CUS
    return max(1, min(most, CUS // tail)) if tail else 1
