"""Sizes of the linear cross entropy (tokens, width, vocabulary) that between them reach every tile side and every way
of cutting its sums, with what is planned for them: checked against the planning code without a GPU, and run on one."""

# sides of the forward tiles, of G's and of the products'; pieces of the vocabulary; ranges of dx's sums in the first piece
# and in the last; ranges of dw's sums; the last piece is shorter where there are several
SIZES = {
    "16": [
        ((2000, 500, 16500), dict(forward=256, grad=256, products=256, pieces=1, ranges=7, last_ranges=7, wranges=1)),
        ((1100, 250, 8001), dict(forward=128, grad=128, products=128, pieces=1, ranges=12, last_ranges=12, wranges=2)),
        ((700, 320, 5000), dict(forward=64, grad=64, products=64, pieces=1, ranges=10, last_ranges=10, wranges=1)),
        ((16400, 512, 20011), dict(forward=256, grad=256, products=256, pieces=2, ranges=1, last_ranges=1, wranges=1)),
        ((16400, 64, 20000), dict(forward=256, grad=256, products=64, pieces=2, ranges=3, last_ranges=3, wranges=4)),
        ((1000, 24, 1154589), dict(forward=256, grad=256, products=64, pieces=5, ranges=63, last_ranges=62, wranges=1)),
    ],
    "f32": [
        ((33, 67, 3), dict(forward=32, grad=32, products=32, pieces=1, ranges=1, last_ranges=1, wranges=1)),
        ((16400, 64, 20000), dict(forward=64, grad=64, products=64, pieces=3, ranges=1, last_ranges=1, wranges=1)),
        ((1000, 8, 392833), dict(forward=64, grad=64, products=64, pieces=3, ranges=63, last_ranges=62, wranges=1)),
    ],
}
