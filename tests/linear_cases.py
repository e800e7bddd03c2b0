"""Sizes of the grouped products that reach each of their kernels, with the kernel they are meant
for: the tile rule's choice is checked against them on the CPU, the results on the GPU.

ROWS: forward, dx and 8-bit products, (tile width, several tiles to a CTA or pair, group sizes,
width of the results, width of the sums).  GRAD_W: (pairs, several, group sizes, in, out).
Groups end inside tiles of every width and inside steps of 16 and 32 columns; some are empty, some
have one row, some several tiles.  Sums end inside a k-block, and the longer ones are of more than
one piece in fp32."""

_FEW = [3, 0, 17, 1, 0, 130, 33, 2]
_130 = [1, 259, 130, 0, 131, 200, 190, 129]
_300 = [650, 0, 1, 511, 300, 449, 289, 200]
_45 = [1 + 37 * q % 89 for q in range(60)]
_5 = [1 + q % 9 for q in range(70)]

ROWS = [
    (32, False, _FEW, 520, 208), (32, True, _5, 1032, 208),
    (64, False, _130, 520, 208), (64, True, _45, 520, 1104),
    (128, False, _300, 520, 1104), (128, True, _45, 2056, 208),
    (256, False, _300, 1032, 208), (256, True, _300, 2056, 1104),
    (256, True, [9001], 2056, 208),
]
GRAD_W = [
    (False, False, _FEW, 200, 520), (False, True, _45, 520, 520),
    (False, True, [77] * 15 + [90], 1032, 520),
    (True, False, _300, 520, 520), (True, True, _300, 1032, 2056), (True, True, _45, 1992, 2048),
]
ROW_IDS = [f"{w}-{len(g)}x{sum(g)}-{i}-{k}" for w, _, g, i, k in ROWS]
GRAD_W_IDS = [f"{'pairs' if p else 'single'}-{len(g)}x{sum(g)}-{i}-{o}" for p, _, g, i, o in GRAD_W]
