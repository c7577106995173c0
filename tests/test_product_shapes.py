"""Which tiles the products over experts take."""
import pytest

from tests.shapes_shim import Shapes


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    return Shapes(str(tmp_path_factory.mktemp("shapes")))


@pytest.mark.parametrize("n,k", [(2048, 4096), (1536, 4096), (4096, 2048), (768, 2048), (1536, 2048), (4096, 7168)])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 6, 8, 16])
def test_experts_without_rows_do_not_count(shapes, rows, n, k):
    """At most as many experts as rows have one: the experts beyond change nothing."""
    few = {shapes.product(rows, e, n, k) for e in range(max(rows, 2), 300)}
    assert len(few) == 1, f"{rows} rows over 2 to 299 experts of {n} x {k} take {few}"


def test_choices(shapes):
    """The measured choices beside the rule."""
    assert shapes.product(4, 64, 2048, 4096) == "64 x 64"      # gated, 4096 x 1024
    assert shapes.product(8, 128, 1536, 2048) == "64 x 64"     # gated, 2048 x 768
    assert shapes.product(8, 32, 4096, 7168) == "128 x 64"     # gated, 7168 x 2048
    assert shapes.product(1023, 0, 2064, 1032) == "128 x 128"  # down
    assert shapes.product(1023, 0, 2064, 2064) == "128 x 64"   # through w1
    assert shapes.product(64, 0, 4096, 2048) == "64 x 64"
    assert shapes.product(8192, 0, 8192, 8192) == "256 x 256"
    assert shapes.weight_grad(8191, 8, 4096, 4096) == "256 x 256"
    assert shapes.weight_grad(2000, 16, 2048, 768) == "128 x 128"
    assert shapes.four_bit(8, 32, 4096) == "16 rows, 4 stages"
    assert shapes.four_bit(128, 32, 4096) == "16 rows, 3 stages"
    assert shapes.four_bit(1, 0, 4096) == "few channels"
    assert shapes.four_bit(300, 4, 100) == "64 rows"


def _row_tiles(counts, n):
    """Heights of the row tiles of 256 channels that the device takes: of 128 to 320 rows at most what the CUs are done
    with first, each expert's of even height in units of 64."""
    channels, best = -(-n // 256), None
    for most in (128, 192, 256, 320):
        tiles = sum(-(-c // most) for c in counts)
        time = (tiles * channels + 255) // 256 * (24 + sum(counts) / tiles)
        if best is None or time < best[0]:
            best = time, most
    heights = set()
    for c in filter(None, counts):
        tiles, units = -(-c // best[1]), -(-c // 64)
        for row in range(tiles):
            heights.add(units // tiles + (row < units % tiles))
    return heights


def test_sizes_of_the_tile_tests(shapes):
    """The GPU tests' sizes choose what they are there for."""
    from tests import test_gpu_product_tiles as T
    for counts, n, k in T.BF16_TILES:
        rows, E = sum(counts) + T.BEFORE + T.BEHIND, len(counts)
        assert shapes.product(rows, E, n, k) == shapes.product(rows, E, n // 64 * 64, k) == "256 x 256"
        assert k // 64 > 2 * 2  # the loop over the two stages goes round
    assert _row_tiles(T.BF16_TILES[0][0], T.BF16_TILES[0][1]) == {1, 2, 3, 4, 5}
    taken = {(shapes.four_bit(M, E, N), K % 128 == 0) for M, E, N, K, _ in T.FOUR_BIT_TILES}
    assert taken >= {(s, words) for s in ("16 rows, 4 stages", "16 rows, 3 stages") for words in (False, True)}


def test_every_tile_has_a_test(shapes):
    """The GPU tests together reach every tile of every product."""
    from tests import test_gpu_ffn as A, test_gpu_matmul_mxfp4 as Q, test_gpu_product_tiles as T
    bf16 = [(M, E, n, k) for M, E, n, k, _ in A.SHAPES]
    bf16 += [(sum(c) + T.BEFORE + T.BEHIND, len(c), n, k) for c, n, k in T.BF16_TILES]
    every = {"64 x 64", "128 x 64", "128 x 128", "256 x 256"}
    assert {shapes.product(*s) for s in bf16} == every                                   # either order, the backward
    assert {shapes.product(M, E, 2 * n, k) for M, E, n, k in bf16[:len(A.SHAPES)]} | {"256 x 256"} == every  # gated
    assert {shapes.weight_grad(*s) for s in bf16} == every
    four = {shapes.four_bit(M, E, N) for M, E, N, *_ in Q.SHAPES + T.FOUR_BIT_TILES}
    assert four == {"few channels", "16 rows, 4 stages", "16 rows, 3 stages", "64 rows"}
