"""Grouped products of small whole numbers, whose sums are exact: the cases of test_gpu_experts_long.py, and inputs in
which any lost, doubled or misplaced row changes the results (test_whole_numbers_cpu.py)."""
import torch

# Sizes that reach each kernel of the gradients of weights (the products n cin cout and the tiles of all groups decide), in
# whole groups and in pieces of groups; y and dx of the same calls go through the large tiles too.
CASES = [("bf16", 1024, 1024, 16, 8000),    # tiles of 256, whole groups
         ("bf16", 264, 520, 2, 60000),      # tiles of 256, pieces
         ("bf16", 256, 256, 70, 65000),     # tiles of 256, pieces, more groups than a wave has lanes
         ("bf16", 512, 512, 70, 31000),     # tiles of 256, whole groups, as many
         ("f32", 512, 512, 20, 9000),       # tiles of 128 in the ring, whole groups
         ("f32", 264, 516, 3, 20000),       # tiles of 128 in the ring, pieces
         ("f32", 128, 128, 70, 125000),     # tiles of 128 in the ring, pieces, more groups than lanes
         ("f32", 512, 256, 70, 20000),      # tiles of 128 in the ring, whole groups, as many
         ("bf16", 515, 1023, 3, 9000),      # tiles of 128 of unaligned rows
         ("bf16", 257, 1023, 3, 20000),
         ("f32", 257, 1023, 3, 11000),
         ("f32", 123, 501, 5, 20384),       # tiles of 64, pieces
         ("bf16", 200, 72, 4, 12345),
         ("f32", 3, 517, 3, 90000)]         # rows shorter than 16 bytes


def inputs(cin, cout, groups, n, gather):
    """x, weight, bias, grad (entries -1, 0, 1, in fp32), offsets with positions of no group at both ends and an empty
    group, and rows of which some are out of range."""
    gen = torch.Generator().manual_seed(31 * cin + cout)
    whole = lambda *s: torch.randint(-1, 2, s, generator=gen, dtype=torch.int8).float()  # noqa: E731
    nx = n // 2 if gather else n
    cuts = torch.sort(torch.randint(5, n - 7, (groups + 1,), generator=gen)).values
    cuts[0], cuts[-1] = 5, n - 7
    if groups > 1:
        cuts[groups // 2 + 1 if groups > 2 else 1] = cuts[groups // 2 if groups > 2 else 0]
    rows = torch.randint(-3, nx + 3, (n,), generator=gen)
    return whole(nx, cin), whole(groups, cout, cin), whole(groups, cout), whole(n, cout), cuts.to(torch.int32), rows.to(torch.int32)
