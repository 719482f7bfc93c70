"""The Python binding's refusals that need tensors on the GPU."""
import pytest
import torch

from stage_software_pipelining_gb300 import build as gemm_build
from stage_software_pipelining_gb300 import quant as Q

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def lib(gpu):
    gemm_build.build()
    return Q.load_library()


class NoTruth:
    def __bool__(self):
        raise TypeError("neither")


def test_arguments_of_no_use_raise_value_errors():
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    q, s = torch.zeros(4, 64, dtype=E4M3, device="cuda"), torch.zeros(4, device="cuda")
    C = torch.zeros(4, 8, dtype=BF16, device="cuda")[:, :4]
    W = q.view(torch.uint8)[:, :32]
    bad = {"gemm_fp8, checked": lambda: Q.gemm_fp8(q, q.t(), C, s, s, checked=NoTruth()),
           "gemv_w4, checked": lambda: Q.gemv_w4(x, W, x[:, :1], C, checked=NoTruth()),
           "stream": lambda: Q.gemv_w4(x, W, x[:, :1], C, stream="1"),
           "eps": lambda: Q.add_rmsnorm(x, x[0], y=x, eps="small")}
    for name, f in bad.items():
        with pytest.raises(ValueError, match="must be"):
            f()
            pytest.fail(f"{name} was accepted")
    torch.cuda.synchronize()
