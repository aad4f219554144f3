"""Rows of the embedding's gradient whose tokens lie in many tiles, of more columns than one block
joins: against the definition in 64 bits, with test_embedding's tolerances."""
import pytest

torch = pytest.importorskip("torch")

from test_embedding import BF16, F32, check_gradient, tokens  # noqa: E402

# tokens, columns, tokens of a tile: 9 and 5 groups of 256 columns, in blocks of 4
CASES = [(3000, 2056, 32), (3000, 1031, 32), (40000, 1104, 64), (40000, 1100, 64), (40000, 1031, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,h,tile", CASES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("by", [0, 1])
def test_rows_of_many_parts_and_many_columns(n, h, tile, dtype, by):
    v = 50
    counts = torch.bincount(tokens(n, v, "zipf", 6).long(), minlength=v)
    assert counts.max() > 17 * tile and counts.min() < 16 * tile  # runs of eight warps, and warps alone
    check_gradient(n, h, v, "zipf", dtype, dtype, by=by, seed=6)
    old = torch.randn(v, h, generator=torch.Generator().manual_seed(7)).to(dtype).cuda()
    check_gradient(n, h, v, "zipf", dtype, dtype, by=by, old=old, seed=6)


@pytest.mark.gpu
@pytest.mark.parametrize("n,h,tile", CASES)
def test_one_row_of_many_parts(n, h, tile):
    check_gradient(n, h, 3, "one", BF16, F32, scale=1.5)
    check_gradient(n, h, 3, "one", F32, BF16, by=1)
