"""Refusals and empty calls of the FFN operators that need no GPU."""
from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G


def test_quantising_no_rows_needs_no_arrays():
    lib = F._library()
    assert lib.gemm_q8_quantize(None, 0, 0, 16, 16, None, 16, None, None) == G.OK
    assert lib.gemm_q8_quantize(None, 0, 1, 16, 16, None, 16, None, None) == G.ERR_INVALID_ARG
    assert lib.gemm_q8_quantize(None, 0, 0, 16, 15, None, 16, None, None) == G.ERR_INVALID_ARG
