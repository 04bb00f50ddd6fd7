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


@pytest.mark.parametrize("colblocks", [False, True])
@pytest.mark.parametrize("rows", [512, 65536])
def test_many_calls_in_a_row(rows, colblocks):
    """Two hundred pairs without a stop, the second call of each with the scale
    given, on what the first has just written over the last pair's."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    codes = torch.empty((rows, 128), dtype=torch.uint8, device="cuda")
    xs = [torch.rand((rows, 256), generator=gen, device="cuda").half() for _ in range(3)]
    g = torch.tensor([0.7], device="cuda")

    def second():
        y = codes.view(torch.float16)
        return (ops.nvfp4_quantize_colblocks if colblocks else ops.nvfp4_quantize)(
            y, tensor_scale=g)[0]

    want = []
    for x in xs:
        ops.nvfp4_quantize(x, codes=codes)
        torch.cuda.synchronize()
        want.append(second())
        torch.cuda.synchronize()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(200):
        ops.nvfp4_quantize(xs[i % 3], codes=codes)
        wrong += (second() != want[i % 3]).sum()
    assert int(wrong) == 0
