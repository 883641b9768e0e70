"""Product shapes that reach every tile form of linear_mx, by the rule that picks them, in both formats."""

# (columns of a tile, on CTA pairs, CTAs that share a tile) -> shapes M, N, K
BY_FORM = {
    (64, False, 1): [(300, 270, 640), (128, 4096, 512), (1, 9216, 1536)],
    (64, False, 2): [(64, 4608, 8960), (300, 1000, 8960), (300, 1536, 8960)],
    (64, False, 4): [(200, 512, 8960), (256, 448, 4192)],
    (64, False, 8): [(1, 64, 8960), (129, 129, 8960), (250, 32, 16384), (1, 32, 1 << 18)],
    (128, False, 1): [(2000, 2048, 96), (100, 12320, 544)],
    (128, True, 1): [(600, 2000, 8960), (1300, 4641, 1568), (1280, 1536, 1536)],
    (192, True, 1): [(2148, 2289, 64), (2148, 2304, 64), (1078, 4872, 768), (5643, 8610, 96)],
    (256, True, 1): [(4096, 4096, 1536), (2500, 8961, 1536), (1280, 8960, 1536), (2000, 2000, 8960)],
}
SHAPES = [s for shapes in BY_FORM.values() for s in shapes]
