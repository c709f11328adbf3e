"""Cases of the expert feed-forward block for every tile size and form of its
products, with the form and tile that each is there for on 256 compute units.

(ranks, experts, capacity, width, hidden, counts), the elements that every
base lies off 16 bytes, and the tile of all six products of both types: "t"
direct loads of the caller's rows, "c" of padded copies, "r" through registers.
"""

CASES = {
    # rows on both sides of a tile, an expert without any, widths that end inside a tile
    "t256": ((2, 4, 3450, 2040, 2032, [[3450, 200, 255, 0], [3450, 57, 0, 0]]), 0),
    "c256": ((2, 4, 3450, 2039, 2041, [[3450, 200, 255, 0], [3450, 57, 0, 0]]), 0),
    "t128": ((1, 5, 4232, 1040, 1032, [[4232, 255, 256, 257, 0]]), 0),
    "c128": ((1, 5, 6232, 1039, 1033, [[6232, 255, 256, 257, 0]]), 0),
    "r128": ((1, 5, 4232, 1040, 1032, [[4232, 255, 256, 257, 0]]), 1),
    "t64": ((2, 4, 300, 264, 200, [[255, 1, 64, 65], [300, 0, 128, 2]]), 0),
    "c64": ((1, 1, 1029, 513, 515, [[1029]]), 0),
    "r64": ((2, 4, 300, 264, 200, [[255, 1, 64, 65], [300, 0, 128, 2]]), 1),
}
