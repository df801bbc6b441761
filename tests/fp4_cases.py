"""Sizes that reach each kernel variant of the 4-bit formats and of the key/value cache on 148 SMs, with the variant.

The rules that choose a variant are host arithmetic (sq_debug_*_plan), so that test_fp4_plans.py checks every entry here
without a GPU: a rule that is changed cannot leave a variant without its test unseen.
"""
from helpers import BF16, F16, F32

# weights as the A operand: (tokens a tile, CTAs a cluster): [(M, N, K), ..]; M > 128: several token tiles
LINEAR_SWAP = {
    (16, 1): [(5, 264, 500)], (16, 2): [(13, 577, 1400)], (16, 4): [(13, 93, 2205)], (16, 8): [(12, 130, 8262)],
    (32, 1): [(23, 570, 124)], (32, 2): [(18, 1379, 1063)], (32, 4): [(29, 289, 2214)], (32, 8): [(21, 119, 3867)],
    (64, 1): [(50, 1000, 300), (77, 4096, 300)], (64, 2): [(64, 1300, 1281), (211, 1331, 1281)],
    (64, 4): [(40, 2000, 2500), (300, 700, 3729)], (64, 8): [(61, 1000, 8200), (250, 200, 6444)],
    (128, 1): [(103, 10303, 198), (128, 20000, 512)], (128, 2): [(65, 4801, 5000), (908, 530, 5000)],
    (128, 4): [(65, 2400, 8000), (1154, 130, 6000)], (128, 8): [(823, 30, 11062)],
}

# CTA pairs, more than two tiles a pair (74 pairs): tile columns: [(M, N, K), ..]; first one whose rows are whole 16-byte
# vectors in every type, then one whose rows are not
LINEAR_PAIRS = {
    256: [(513, 18944, 287), (513, 18879, 287), (257, 21504, 1100)],
    192: [(257, 19072, 600), (257, 18975, 1000)],
    128: [(513, 9472, 1000), (513, 9469, 1000)],
}

# quantisers: type, rows, K, columns between rows, bytes an access, rows a thread, at least so many units a block.  The
# last scale tile holds 1, 9, 33, 127 or all rows; K ends inside a block and a scale tile, or at the end of one.
QUANT = [
    (F16, 1153, 1504, 0, 32, 4, 1), (BF16, 1161, 1555, 5, 16, 4, 1), (BF16, 1185, 1300, 12, 32, 4, 1),
    (F16, 2303, 4100, 12, 32, 4, 2), (BF16, 2304, 4088, 0, 16, 4, 2), (BF16, 2300, 4101, 0, 0, 1, 2),
    (F32, 1153, 7700, 0, 16, 4, 2), (F32, 2057, 4712, 0, 32, 4, 2), (F32, 2303, 4100, 4, 32, 4, 2),
    (F32, 2300, 4101, 0, 0, 1, 2), (F32, 2210, 520, 0, 32, 1, 2),
]

# dequantiser: output type, rows, K, bytes an access, rows a thread, at least so many units a block
VALUES = [
    (F16, 1153, 1504, 32, 4, 1), (BF16, 1161, 1560, 16, 4, 1), (BF16, 2303, 4112, 32, 4, 2), (F16, 2304, 4104, 16, 4, 2),
    (BF16, 2300, 4101, 0, 1, 2), (F32, 2303, 4104, 32, 4, 2), (F32, 2303, 4100, 16, 4, 2), (F32, 2300, 4101, 0, 1, 2),
]

# cache writes: tokens, H, D, steps a warp, chunks a lane
KV_WRITES = [(5001, 8, 128, 2, 1), (7603, 5, 80, 2, 1), (9601, 1, 500, 2, 1), (5001, 8, 64, 1, 1), (3001, 3, 600, 1, 2)]

# cache reads: rows, H, D, warps a token (0: rows laid end to end)
KV_READS = [(2501, 8, 128, 1), (2501, 32, 128, 1), (2400, 24, 64, 1), (2500, 3, 600, 1), (300, 32, 128, 8), (600, 24, 128, 4),
            (1200, 8, 128, 2), (2501, 5, 128, 0), (2501, 7, 100, 0)]
