"""The host quantiser of fp8 weights on values that are not finite."""
import numpy as np

from int4_routed_expert_gemv_b200 import quantize as Q


def test_blocks_that_are_not_finite():
    rng = np.random.default_rng(1)
    W = rng.standard_normal((256, 300)).astype(np.float32)
    want, ws = Q.quantize_matrix_fp8(W)
    W[5, 7] = np.nan                 # block (0, 0)
    W[130, 130], W[131, 140] = np.inf, -np.inf      # block (1, 1)
    q, s = Q.quantize_matrix_fp8(W)
    assert np.isnan(s[0, 0]) and (q[:128, :128] & 0x7F == 0x7F).all()
    assert s[1, 1] == np.inf
    block = q[128:, 128:256] & 0x7F
    assert block[2, 2] == 0x7F and block[3, 12] == 0x7F and (block != 0).sum() == 2
    # the other blocks are what they were
    for i in range(2):
        for j in range(3):
            if (i, j) not in ((0, 0), (1, 1)):
                at = np.s_[i * 128:i * 128 + 128, j * 128:j * 128 + 128]
                assert s[i, j] == ws[i, j] and np.array_equal(q[at], want[at])
