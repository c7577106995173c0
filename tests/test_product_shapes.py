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
