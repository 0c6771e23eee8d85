"""The block-scaled product at the 8B configuration's largest shapes, and at sizes on both sides of
its rules for tiles and splits, against a 64-bit product on the GPU."""
import pytest

from cached_masked_decoding_gb300 import binding
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_cuda()
    binding.lib()
    return t


def values(torch, codes, scales):
    """codes [rows][K] and bytes [ceil(K/128)][rows] to float64."""
    e = torch.exp2(scales.double() - 127).t().repeat_interleave(128, dim=1)[:, :codes.shape[1]]
    return codes.view(torch.float8_e4m3fn).double() * e


SHAPES = [
    # M, N, K
    (4096, 1, 12288), (4096, 32, 12288), (4096, 2048, 12288),                 # the down projection
    (126464, 1, 4096), (126464, 32, 4096), (126464, 129, 4096),               # the LM head
    (24576, 33, 4096), (12288, 2048, 4096),
    (4096, 65, 4096), (4096, 192, 4096), (4096, 193, 4096), (4095, 401, 4096), (129, 3001, 1552), (20000, 385, 16),
]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_of_large_shapes(torch, M, N, K, out):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)
    kb = -(-K // 128)

    def operand(rows):
        c = torch.randint(0, 0x7f, (rows, K), generator=g, device="cuda", dtype=torch.uint8)
        c |= torch.randint(0, 2, (rows, K), generator=g, device="cuda", dtype=torch.uint8) << 7
        return c, torch.randint(117, 123, (kb, rows), generator=g, device="cuda", dtype=torch.uint8)

    (w, ws), (x, xs) = operand(M), operand(N)
    y = torch.full((N + 1, M), 3.0, device="cuda", dtype=torch.float32 if out == "f32" else torch.bfloat16)
    binding.op_gemm8(w.data_ptr(), ws.data_ptr(), x.data_ptr(), xs.data_ptr(), y.data_ptr(), out, M, N, K)
    assert binding.op_check() == 0
    assert (y[N] == 3.0).all()
    xv = values(torch, x, xs)
    half = 2.0 ** -24 if out == "f32" else 2.0 ** -8
    # products of codes are exact; a float32 sum of 32 products a step, rounded or cut to 24 bits: K/32 steps and
    # the joined parts
    steps = K // 32 + 16
    for m0 in range(0, M, 8192):
        wv = values(torch, w[m0:m0 + 8192], ws[:, m0:m0 + 8192])
        want = xv @ wv.t()
        tol = steps * 2.0 ** -23 * (xv.abs() @ wv.abs().t()) + half * want.abs()
        assert ((y[:N, m0:m0 + 8192].double() - want).abs() <= tol).all()
