"""Shapes (m, n, k) of the 8-bit product, one at least for every way that plan_product8 lays a product out
(tests/test_product_cases_cpu.py checks that): the kernel of few rows by its row blocks, tiles of 64, 128 and 256, each
whole or with k split, with one tile a workgroup or several, and the last rows apart with every kind of plan for them.
No size is a multiple of 16."""

# for fp32 results, bf16 ones with fp32 sums, and bf16 ones with cut sums; a scale a column or a tile of b
EVERY = [(1, 63, 333), (33, 1635, 333), (69, 1375, 333), (69, 2121, 333), (69, 63, 8149), (137, 747, 31281),
         (16855, 63, 13293), (33595, 137, 333), (33595, 69, 333), (69, 1155, 15021), (69, 2749, 24497), (33595, 69, 4419),
         (25939, 69, 547), (16855, 69, 701), (47427, 137, 547)]
# for bf16 results with cut sums and a scale for each tile of b
CUT_TILES = [(39917, 137, 701), (56351, 259, 1147), (137, 4237, 16977), (137, 4237, 45139), (47427, 525, 793),
             (33595, 889, 4995), (51697, 525, 4995), (33595, 815, 547), (21831, 1375, 2707), (21831, 1375, 427),
             (28275, 525, 547), (36619, 259, 4995), (47427, 259, 4995), (51697, 403, 9209), (33595, 309, 1297),
             (33595, 309, 2119), (21831, 525, 547), (33595, 259, 793), (47427, 137, 333), (7755, 6525, 21677), (33595, 1059, 9209),
             (2121, 8453, 21677)]
