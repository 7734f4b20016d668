"""Sizes of the cross entropy's and the gated product's gradients, each with the way it stands for; test_layer_pieces_host.py
holds them to it without a GPU, test_layer_pieces_gpu.py runs them."""

#: (T, I, V, pieces of the vocabulary, parts of grad_x in a piece): the carry of grad_x's sums across pieces, one part (the
#: last piece scales and rounds) and several (each carried for itself), shorter last pieces, rows on and off 16 bytes
PIECES = [(7000, 48, 20011, 2, 2), (7000, 520, 20011, 2, 1), (7001, 16, 39000, 3, 2), (3001, 72, 50021, 2, 4),
          (20000, 328, 30011, 2, 1), (2100, 15, 70001, 2, 5), (17000, 336, 20011, 2, 1)]

#: (T, I, V, pieces, parts, blocks of the last piece): fewer blocks in the last piece than there are parts
SHORT = (7000, 8, 5895169, 304, 2, 1)

#: (T, I, F): grad_w by rows, at least a tile for every pair of CTAs, I a multiple of 16 but for the first two not of 256,
#: ragged ends in both directions, T on and off whole blocks, the last one more than 16384 tokens in two runs
BY_ROWS = [(130, 1040, 2100), (17, 2048, 1290), (1, 1536, 1700), (64, 3088, 900), (700, 1040, 2049), (16500, 1040, 2100)]

#: (T, I, F, the way): grad_w of more than 16384 tokens with its values on the lanes, the runs one after the other ("pair") or
#: as tiles of their own ("apart"), tiles of both widths, rows on and off 16 bytes
RUNS = [(16500, 1279, 2100, "pair"), (16500, 520, 2100, "apart"), (33000, 264, 2100, "apart"), (16500, 1279, 1300, "apart")]
