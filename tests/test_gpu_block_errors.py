"""An error that a call of the transformer-block operators meets is reported by that call and by
no later one.

The error is made on the host: a stream whose capture has been invalidated refuses every launch
until the capture is ended, and nothing of the call reaches the GPU."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

RELAXED = 2


class _BrokenCapture:
    """A stream that refuses launches while the context is open."""

    def __enter__(self):
        self.cu = ctypes.CDLL("libcuda.so.1")
        self.stream = torch.cuda.Stream()
        handle = ctypes.c_void_p(self.stream.cuda_stream)
        assert self.cu.cuStreamBeginCapture_v2(handle, RELAXED) == 0
        assert self.cu.cuStreamSynchronize(handle) != 0   # not allowed there: ends the capture's use
        self.ctx = torch.cuda.stream(self.stream)
        self.ctx.__enter__()
        return self

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)
        graph = ctypes.c_void_p()
        self.cu.cuStreamEndCapture(ctypes.c_void_p(self.stream.cuda_stream), ctypes.byref(graph))


def _calls(gs):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda")
    X, S = mk(64, 96), mk(96)
    Y, M, I = gs.gs_layer_norm(X, S)
    calls = {"layer_norm": lambda: gs.gs_layer_norm(X, S),
             "layer_norm_backward": lambda: gs.gs_layer_norm_backward(Y, X, S, M, I),
             "dropout": lambda: gs.gs_dropout(X, 0.5, 1, 2)}
    m, rows = gs.gs_relative_buckets((1, 90), (1, 90), 8, 32)
    one, one_rows = gs.gs_relative_buckets((1, 1), (1, 90), 8, 32)
    for name, dt in (("fp32", torch.float32), ("fp16", torch.float16), ("bf16", torch.bfloat16)):
        Q, K, V, dO = (mk(2, 90, 2, 64).to(dt) for _ in range(4))
        t, t1 = mk(rows, 2).to(dt), mk(one_rows, 2).to(dt)
        O, L = gs.gs_attention(Q, K, V, t, m)
        few, none = Q[:, :1].contiguous(), Q[:, :0]
        calls.update({
            f"few_{name}": lambda few=few, K=K, V=V, t1=t1: gs.gs_attention(few, K, V, t1, one),
            f"attention_{name}": lambda Q=Q, K=K, V=V, t=t: gs.gs_attention(Q, K, V, t, m),
            f"no_bias_{name}": lambda Q=Q, K=K, V=V: gs.gs_attention(Q, K, V),
            f"backward_{name}": lambda dO=dO, Q=Q, K=K, V=V, O=O, L=L, t=t:
                gs.gs_attention_backward(dO, Q, K, V, O, L, t, m),
            f"no_query_{name}": lambda none=none, K=K, V=V, L=L: gs.gs_attention_backward(
                none, none, K, V, none, L[:, :, :0].contiguous())})
    return calls


def test_an_error_stays_with_its_call(gs_cuda):
    calls = _calls(gs_cuda)
    torch.cuda.synchronize()
    wrong = []
    for name, call in calls.items():
        with _BrokenCapture():
            try:
                call()
                wrong.append(f"{name}: no error on a stream that refuses it")
            except gs_cuda.GsError as e:
                assert e.status == 7, e
        for after in ("layer_norm", "dropout"):
            try:
                calls[after]()
            except gs_cuda.GsError as e:
                wrong.append(f"{name} left an error to {after}: {e}")
    torch.cuda.synchronize()
    assert not wrong, wrong
    assert gs_cuda.gs_device_status() == 0
