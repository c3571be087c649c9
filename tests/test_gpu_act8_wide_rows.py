"""GPU tests of 8-bit activations in single rows whose byte offsets pass 31 and
32 bits: the same bits as the row cut into short ones.  What is restored lies in
the second half of a buffer whose first half stays as it was."""
import pytest
import torch

import thread_register_tile_amd as trt

pytestmark = pytest.mark.gpu

SHORT = 1 << 15     # columns, a multiple of a scale's 32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    trt.lib()


@pytest.mark.parametrize("dtype,cols", [(torch.float32, (1 << 29) + 3 * SHORT + 37), (torch.float32, 1 << 30),
                                        (torch.bfloat16, (1 << 30) - 3), (torch.float16, 1 << 30)])
def test_one_row(dtype, cols):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, cols, device="cuda", generator=gen, dtype=dtype)
    q, scale = trt.act8_pack(x)
    whole = cols // SHORT * SHORT
    pieces = [(slice(0, whole), (-1, SHORT))] + ([(slice(whole, cols), (1, -1))] if whole < cols else [])
    buf = torch.full((2 * cols,), 77.0, device="cuda", dtype=dtype)
    out = buf[cols:].view(1, cols)
    trt.act8_unpack(q, scale, dtype, out=out)
    for part, shape in pieces:
        q1, s1 = trt.act8_pack(x[0, part].view(shape))
        assert torch.equal(q[0, part].view(q1.shape), q1)
        assert torch.equal(scale[0, part.start // 32:-(-part.stop // 32)].view(s1.shape), s1)
        assert torch.equal(out[0, part].view(q1.shape), trt.act8_unpack(q1, s1, dtype))
    assert bool((buf[:cols] == 77).all())
