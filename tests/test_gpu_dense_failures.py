"""A launch of the dense sublayer that fails on the host leaves nothing behind: the next call on the thread, of
the dense sublayer or of the routed block, runs as if it had not been.

The failure: a capture that a synchronisation has invalidated refuses every launch on its stream.  Nothing
reaches the GPU."""
import ctypes
import threading

import pytest
import torch

import test_gpu_fp8 as t8
import test_gpu_gated_ffn as tg

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


class Invalidated:
    """A stream in a capture that is no longer valid (relaxed mode: allocations are allowed)."""

    def __enter__(self):
        self.rt = ctypes.CDLL(f"libcudart.so.{torch.version.cuda.split('.')[0]}")
        self.stream = torch.cuda.Stream()
        self.handle = ctypes.c_void_p(self.stream.cuda_stream)
        torch.cuda.synchronize()
        assert self.rt.cudaStreamBeginCapture(self.handle, 2) == 0
        assert self.rt.cudaStreamSynchronize(self.handle) == 900  # not permitted under capture: it ends the capture
        self.rt.cudaGetLastError()  # PyTorch's copy of the runtime forgets it, the library has its own
        return self.stream

    def __exit__(self, *_):
        graph = ctypes.c_void_p()
        assert self.rt.cudaStreamEndCapture(self.handle, ctypes.byref(graph)) == 901 and not graph.value
        self.rt.cudaGetLastError()


def calls():
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(0)
    w = torch.ones(256, device="cuda")
    few, many = tg.make(2, 256, 264, BF16), tg.make(150, 256, 264, BF16)
    saved = m.gated_ffn(*many[:4], save=True)[1]
    a, sa = t8.operand(150, 256, 1, torch.float8_e4m3fn, gen)
    b, sb = t8.operand(264, 256, 128, torch.float8_e4m3fn, gen)
    x, dy = many[0], many[4]
    return {
        "block_norm": lambda st: list(m.block_norm(x, norm_next=w, stream=st))[1:],
        "block_norm_backward": lambda st: list(m.block_norm_backward(x, norm_next=w, d_y=dy, stream=st).values()),
        "gated_ffn, two rows": lambda st: [m.gated_ffn(*few[:4], stream=st)],
        "gated_ffn": lambda st: [m.gated_ffn(*many[:4], stream=st)],
        "gated_ffn_backward": lambda st: list(m.gated_ffn_backward(*many[:4], saved, dy, stream=st).values()),
        "fp8_matmul, two rows": lambda st: [m.fp8_matmul(a[:2], sa[:2], b, sb, stream=st)],
        "fp8_matmul": lambda st: [m.fp8_matmul(a, sa, b, sb, stream=st)],
        "fp8_quantise": lambda st: [t.view(torch.uint8) for t in m.fp8_quantise(x, stream=st)],
    }


def in_a_thread(work):
    """Runs work in a thread of its own: what the CUDA runtime recorded for it ends with it, also where the test fails."""
    failed = []

    def run():
        try:
            work()
        except BaseException as e:
            failed.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if failed:
        raise failed[0]


@pytest.mark.parametrize("which", ["block_norm", "block_norm_backward", "gated_ffn, two rows", "gated_ffn",
                                   "gated_ffn_backward", "fp8_matmul, two rows", "fp8_matmul", "fp8_quantise"])
def test_a_failed_launch_is_reported_once(cuda_lib, which):
    import deepseek_v4_moe_gb300 as m
    from deepseek_v4_moe_gb300 import _lib

    def work():
        all_calls = calls()
        want = {k: f(None) for k, f in all_calls.items()}
        with Invalidated() as st:
            with pytest.raises(m.MoeFFNError) as e:
                all_calls[which](st)
            assert e.value.code == _lib.ERR_CUDA and "launch" in str(e.value)
        for k, f in all_calls.items():
            assert all(torch.equal(a, b) for a, b in zip(f(None), want[k])), k
        assert m.dense_status() == 0

    in_a_thread(work)


def test_the_routed_block_after_a_failed_launch(cuda_lib):
    import synth
    from deepseek_v4_moe_gb300 import MoeFFN, MoeFFNError, config_from
    from synth.device import upload

    def work():
        cfg = synth.CONFIGS["c0_tiny"]
        dev = upload(synth.Case(cfg), "cuda:0")
        h = MoeFFN(config_from(cfg), {cfg.layer: dev["weights"]})
        want = h.forward(dev["state"], dev["token_ids"], cfg.layer).clone()
        f = calls()["gated_ffn"]
        f(None)
        with Invalidated() as st:
            with pytest.raises(MoeFFNError):
                f(st)
        assert torch.equal(h.forward(dev["state"], dev["token_ids"], cfg.layer), want) and h.status() == 0
        h.close()

    in_a_thread(work)
