"""Host-side test of the bfloat16 products' rule: rows of D that are no whole vectors
cost the two-SM tiles nothing more, so that such products take them where their
aligned neighbours do.  Measured on GB300 (us, small tiles of 128 rows and two-SM
tiles): 5576 x 71 x 3154 42.5 and 23.9, 1463 x 72 x 4959 21.7 and 14.4, weight
gradient 1514 x 90 x 4094 16.7 and 11.6."""

import pytest

from dense_int8_matrix_gb300 import binding as B
from dense_int8_matrix_gb300 import build as build_mod


@pytest.mark.parametrize("m,k,n,form", [(5576, 71, 3154, B.GEMM_FORM_NT), (1463, 72, 4959, B.GEMM_FORM_NT), (1514, 90, 4094, B.GEMM_FORM_TN),
                                        (5497, 214, 430, B.GEMM_FORM_NT)])
def test_ragged_rows_take_the_tile_of_aligned_ones(m, k, n, form):
    build_mod.build()
    for ragged in (n, (n + 7) // 8 * 8):
        p = B.gemm_bf16_linear_plan_for_sms(m, k, ragged, 152, form)
        assert (p.path, p.bm, p.bn, p.split_k) == (B.GEMM_PATH_TENSOR, 256, 256, 1), ragged
