"""What the dense sublayer's Python functions answer to arguments that are no tensors, with a stream and without:
TypeError, as documented.  No GPU: nothing gets that far."""
import pytest
import torch

import deepseek_v4_moe_gb300 as m

CPU = torch.zeros(2, 8)


class Stream:
    """Has what a stream of the GPU has that is looked at before the tensors are."""
    device = torch.device("cuda:0")


@pytest.mark.parametrize("stream", [None, Stream()])
@pytest.mark.parametrize("bad", [None, 3, [[1.0]]])
def test_no_tensor(bad, stream):
    for call in (lambda: m.block_norm(bad, norm_next=CPU, stream=stream),
                 lambda: m.block_norm_backward(bad, norm_next=CPU, d_y=CPU, stream=stream),
                 lambda: m.gated_ffn(bad, CPU, CPU, CPU, stream=stream),
                 lambda: m.gated_ffn_backward(bad, CPU, CPU, CPU, (CPU, CPU), CPU, stream=stream),
                 lambda: m.fp8_quantise(bad, stream=stream), lambda: m.fp8_matmul(bad, CPU, CPU, CPU, stream=stream)):
        with pytest.raises(TypeError):
            call()


def test_tensors_of_another_device_than_the_stream():
    for call in (lambda s: m.gated_ffn(CPU, CPU, CPU, CPU, stream=s), lambda s: m.fp8_quantise(CPU, stream=s),
                 lambda s: m.block_norm(CPU, norm_next=CPU, stream=s)):
        for stream in (None, Stream()):
            with pytest.raises(ValueError):
                call(stream)
