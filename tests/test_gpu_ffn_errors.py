"""An error that an earlier call of the caller's left behind in the HIP runtime
is neither reported as an operator's own nor taken away."""
import pytest
import torch

from tensor_gemm_reduce_lds_amd import ffn as F

from gpu_util import say

pytestmark = pytest.mark.gpu


def test_an_older_error_of_the_caller_is_not_reported():
    hip = F._library()                       # (its runtime's functions resolve through it)
    s = torch.cuda.current_stream()
    bf = lambda *n: torch.randn(n, device="cuda").bfloat16()  # noqa: E731
    x, y, w = bf(6, 64), bf(6, 64), torch.ones(64, device="cuda")
    q, sq = torch.empty((6, 64), dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    b, c, dw = bf(2, 64, 64), bf(6, 64), bf(2, 64, 64)
    o = [bf(6, 64) for _ in range(4)] + [torch.empty((2, 64), device="cuda")]
    norm = F.BlockNormPlan(6, 64, backward=1)
    long_norm = F.BlockNormPlan(6, 16384, backward=1)      # (its sums lie in LDS)
    xl, wl = bf(6, 16384), torch.ones(16384, device="cuda")
    ol = [bf(6, 16384) for _ in range(4)] + [torch.empty((2, 16384), device="cuda")]
    q8, q8_tile = F.Q8Plan(6, 64, 64), F.Q8Plan(70, 64, 64)
    q70, sq70, d70 = torch.zeros((70, 64), dtype=torch.int8, device="cuda"), torch.ones(70, device="cuda"), bf(70, 64)
    nn, tn = F.GroupedPlan(6, 64, 64, 2, F.GROUPED_NN), F.GroupedPlan(6, 64, 64, 2, F.GROUPED_TN)
    odd = F.GroupedPlan(6, 63, 64, 2, F.GROUPED_NN, ldb=64, ldc=64)
    wq, sw = torch.zeros((64, 64), dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    calls = {
        "forward": lambda: norm.run(x, y, w, None, w, o[0], o[1], stream=s),
        "backward": lambda: norm.backward(x, x, x, y, w, None, w, o[2], o[3], o[4][0], None, o[4][1], stream=s),
        "backward, no rows": lambda: norm.backward(x, x, x, y, w, None, w, o[2], o[3], o[4][0], None, o[4][1], rows=0, stream=s),
        "backward, long": lambda: long_norm.backward(xl, xl, xl, xl, wl, None, wl, ol[2], ol[3], ol[4][0], None, ol[4][1], stream=s),
        "quantize": lambda: F.q8_quantize(x, q, sq, 6, 64, stream=s),
        "q8 rows": lambda: q8.run(q, sq, wq, sw, None, c, stream=s),
        "q8 tile": lambda: q8_tile.run(q70, sq70, wq, sw, None, d70, stream=s),
        "grouped": lambda: nn.run(x, b, off, c, stream=s),
        "grouped gradient": lambda: tn.run(x, y, off, dw, stream=s),
        "grouped odd": lambda: odd.run(x, b, off, c, stream=s),
    }
    for name, call in calls.items():
        say("older error:", name)
        torch.cuda.synchronize()
        left = hip.hipSetDevice(1 << 20)
        assert left != 0 and hip.hipPeekAtLastError() == left
        try:
            call()
            assert hip.hipPeekAtLastError() == left, name
        finally:
            hip.hipGetLastError()
        call()
        assert hip.hipPeekAtLastError() == 0, name
    torch.cuda.synchronize()
