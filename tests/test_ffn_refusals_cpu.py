"""Refusals and empty calls of the FFN operators that need no GPU."""
import pytest

from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G


def test_quantising_no_rows_needs_no_arrays():
    lib = F._library()
    assert lib.gemm_q8_quantize(None, 0, 0, 16, 16, None, 16, None, None) == G.OK
    assert lib.gemm_q8_quantize(None, 0, 1, 16, 16, None, 16, None, None) == G.ERR_INVALID_ARG
    assert lib.gemm_q8_quantize(None, 0, 0, 16, 15, None, 16, None, None) == G.ERR_INVALID_ARG


class _Offsets:
    """A stand-in for a tensor on the GPU."""

    def __init__(self, n=4, size=4, floating=False, cuda=True, contiguous=True):
        self.n, self.size, self.floating, self.is_cuda, self.contiguous = n, size, floating, cuda, contiguous

    def numel(self):
        return self.n

    def element_size(self):
        return self.size

    def is_floating_point(self):
        return self.floating

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return 4096


@pytest.mark.parametrize("kw,ok", [(dict(), True), (dict(n=9), True), (dict(size=8), False), (dict(floating=True), False),
                                   (dict(n=3), False), (dict(cuda=False), False), (dict(contiguous=False), False)], ids=str)
def test_offsets_of_another_layout_are_refused(kw, ok):
    """Nothing may reach the library with them: its call is replaced here."""
    plan, calls = object.__new__(F.GroupedPlan), []
    plan.handle, plan._rows, plan._offsets = None, 8, 4
    plan._run = lambda *a: calls.append(a) or G.OK
    if ok:
        plan.run(None, None, _Offsets(**kw), None)
    else:
        with pytest.raises(G.GemmRsError) as e:
            plan.run(None, None, _Offsets(**kw), None)
        assert e.value.code == G.ERR_INVALID_ARG
    assert len(calls) == int(ok)
    plan.run(None, None, 4096, None)
    assert len(calls) == 1 + int(ok)


def test_offsets_may_be_anything_that_has_an_address():
    class Address:
        def data_ptr(self):
            return 4096

    plan, calls = object.__new__(F.GroupedPlan), []
    plan.handle, plan._rows, plan._offsets = None, 8, 4
    plan._run = lambda *a: calls.append(a) or G.OK
    plan.run(None, None, Address(), None)
    assert calls[0][3] == 4096


def test_rows_whose_last_steps_pass_32_bits_are_unsupported():
    """Steps of 64 rows are counted in 32 bits, a few past the last one: with 2^31
    - 1 rows of one expert the end of the last step would be negative."""
    for m, want in ((2 ** 31 - 1, G.ERR_UNSUPPORTED), (2 ** 31 - 1024, G.ERR_UNSUPPORTED)):
        with pytest.raises(G.GemmRsError) as e:
            F.GroupedPlan(m, 8, 8, 1, F.GROUPED_TN)
        assert e.value.code == want
    most = 2 ** 31 - 1025
    assert (-(-most // 64) + 4) * 64 < 2 ** 31
