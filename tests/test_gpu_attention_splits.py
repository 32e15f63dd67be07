"""Every split of the key sweep's work: how many waves deal a tile's queries among themselves goes by the number of tiles of 32
keys times key heads, and by the query tiles there are for one (group heads x mean length / 64)."""
import pytest

from test_gpu_attention import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_buckets", [0, 16])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lens,hq,hk", [
    ([300, 200], 4, 1),      # 17 tiles: eight waves, or as many as registers and LDS hold (128 wide: four, float32 with a bias two)
    ([150] * 20, 8, 4),      # 452 tiles of 4 items: four waves
    ([150] * 20, 8, 8),      # 904 tiles of 2 items: two waves
    ([70] * 30, 6, 3),       # 285 tiles of 2 items: two waves
    ([100, 20] * 20, 4, 4),  # 460 tiles of less: one wave
])
def test_waves_of_a_tile_of_keys(lens, hq, hk, d, dtype, n_buckets):
    check(lens, hq, hk, d, dtype, n_buckets=n_buckets)


@pytest.mark.parametrize("n_buckets,dtype,d", [(0, "bf16", 128), (16, "bf16", 64), (0, "f32", 32)])
def test_more_tiles_than_the_card_holds(n_buckets, dtype, d):
    """6,552 tiles of 4 items: one wave; 2,184: two."""
    check([260] * 30, 24, 24, d, dtype, n_buckets=n_buckets)
    check([260] * 30, 8, 8, d, dtype, n_buckets=n_buckets)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[2000] + [3] * 100, [3] * 300 + [1500]])
def test_one_long_sequence_among_short_ones(lens, dtype):
    """The splits go by the mean length: few waves for the long one's tiles, right all the same."""
    check(lens, 2, 1, 64, dtype, n_buckets=16)
