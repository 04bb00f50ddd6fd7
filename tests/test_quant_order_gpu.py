"""A quantiser call whose input is the output of the call right before it in
the stream: it reads what that call has written, whenever its kernels are
scheduled."""
import pytest
import torch

from bit_quantization_b200 import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("had", [False, True])
@pytest.mark.parametrize("rows,cols", [(37, 256), (4096, 256), (65536, 256)])
def test_codes_of_the_previous_call_as_input(rows, cols, had, given):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device="cuda")
    # values without a sign have codes 0 to 7, of which no two bytes are an
    # fp16 infinity or NaN
    xs = [torch.rand((rows, cols), generator=gen, device="cuda").half() for _ in range(6)]
    g = torch.tensor([0.7], device="cuda") if given else None
    got = []
    for x in xs:
        ops.nvfp4_quantize(x, codes=codes)
        got.append(ops.nvfp4_quantize(codes.view(torch.float16), use_hadamard=had,
                                      tensor_scale=g))
    torch.cuda.synchronize()
    for x, y in zip(xs, got):
        ops.nvfp4_quantize(x, codes=codes)
        torch.cuda.synchronize()
        want = ops.nvfp4_quantize(codes.view(torch.float16), use_hadamard=had,
                                  tensor_scale=g)
        torch.cuda.synchronize()
        for a, b in zip(want, y):
            assert torch.equal(a, b)
