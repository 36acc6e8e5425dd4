"""Shapes that reach every tile of the many-row MX FP4 products on 256 compute
units, with ragged edges both ways.  K is chosen apart: how a row's scales and
activations are aligned picks the variant of a tile."""

#: tile of csrc/mx_plan.hpp -> (M, N)
W4A4 = {
    "k32x64": [(90, 5003), (511, 1023)],
    "k64x64": [(63, 13313), (500, 2047)],
    "k128x128": [(700, 3333), (129, 13441)],
    "k256x256": [(2047, 6401), (1025, 9985)],
}
W4A16 = {
    "k32x64": [(90, 5003), (33, 8191)],
    "k64x64": [(63, 13313), (500, 2047)],
    "k64x128": [(500, 4001), (65, 13317)],
    "k128x128": [(300, 13001), (1025, 4100)],
    "kLarge": [(1290, 6401), (900, 4001)],   # whole tiles and quarters; quarters alone
}

#: columns: several stages and a last one that is short or, over groups of
#: waves, missing.  Blocks a row: a multiple of 16, of 4, of neither.
K_W4A4 = {"scales by 16": 1536, "scales by 12": 1504, "short": 40, "odd": 2077}
K_W4A16 = {"scales by 16": 1536, "scales by 4": 1408, "scales by 1": 1432, "rows anywhere": 1429, "short": 40,
           "odd": 37}


def large_w4a4(K, yt):
    """Whether 256 x 256 tiles are allowed: not for f32 results with scales at any address."""
    return yt == "bf16" or -(-K // 32) % 16 == 0


def variants_w4a4():
    """(tile, scales by 16 bytes, result type) that pick() in mx_tiled_w4a4.hip can choose."""
    return {(t, s, yt) for t in W4A4 for s in (False, True) for yt in ("f32", "bf16")
            if (t in ("k128x128", "k256x256") or not s) and (t != "k256x256" or s or yt == "bf16")}


def tile_w4a4(tile, K, yt):
    return "k128x128" if tile == "k256x256" and not large_w4a4(K, yt) else tile


def variant_w4a4(tile, K, yt):
    tile = tile_w4a4(tile, K, yt)
    return tile, tile in ("k128x128", "k256x256") and -(-K // 32) % 16 == 0, yt


def variants_w4a16():
    """(tile, activation rows on 16 bytes, bytes of a row's scales a load) of mx_tiled_w4a16.hip."""
    small = {(t, x, s) for t in W4A16 if t != "kLarge" for x, s in ((True, 4), (True, 1), (False, 1))}
    return small | {("kLarge", True, 16), ("kLarge", True, 4)}


def large_w4a16(K):
    return K % 8 == 0 and -(-K // 32) % 4 == 0


def variant_w4a16(tile, K):
    B = -(-K // 32)
    if tile == "kLarge":
        return tile, True, 16 if B % 16 == 0 else 4
    return tile, K % 8 == 0, 4 if large_w4a16(K) else 1


def cases_w4a4():
    for tile, shapes in W4A4.items():
        for i, (M, N) in enumerate(shapes):
            for K in list(K_W4A4.values())[:2 if i else None]:
                yield tile, M, N, K


def cases_w4a16():
    for tile, shapes in W4A16.items():
        for i, (M, N) in enumerate(shapes):
            for K in list(K_W4A16.values())[:4 if i else None]:
                if tile != "kLarge" or large_w4a16(K):
                    yield tile, M, N, K
