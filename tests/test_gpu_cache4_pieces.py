"""Units of the 4-bit decode cut into every number of pieces around where the
merge changes its form: up to 4 by a warp, up to 16 by the CTA, more of them
in groups of 8."""

import pytest

from test_gpu_fp4 import assert_lse, assert_out, decode_case, expected, run_decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,D,dtype", [(1, 64, "fp16"), (4, 128, "bf16"), (8, 128, "fp16"), (8, 64, "bf16")])
@pytest.mark.parametrize("ctas", [1, 3, 4, 5, 7, 8, 9, 15, 16, 17, 18, 24, 25, 33])
def test_number_of_pieces(cuda_device, G, D, dtype, ctas):
    # one unit over all the CTAs (a granule is 128 tokens), then two, of which one CTA holds an end of each
    for lens in ([260 * ctas], [150 * ctas, 130 * ctas]):
        c = decode_case([G, D, ctas], lens, G, 1, D, 16, dtype)
        out, lse, _, tol, _ = expected(c)
        got, norm, st = run_decode(c, cuda_device, ctas)
        assert st == 0
        assert_out(got, out, tol, dtype)
        assert_lse(norm, lse, c)
