"""Layers of two shapes driven from several host threads at once, each on its
own stream with its own buffers: every call is accepted and gives the bits of
a call alone. Kernels that take their shared memory at launch serve both
shapes with one instance, whose limit the threads share."""
import ctypes
import math
import threading

import pytest
import torch

from windowed_attention_b200.layer import RibLayer
from windowed_attention_b200.workloads import LayerShape, make_inputs

pytestmark = pytest.mark.gpu

SHAPES = [LayerShape(B=1, H=32, W=32, C=48, heads=3, R=16, L=10, hidden=64, window=16),
          LayerShape(B=1, H=32, W=48, C=180, heads=6, R=16, L=10, hidden=64, window=16)]


def _layer(shape):
    inp = make_inputs("train", layer=shape)
    X = torch.randn(shape.B, shape.H, shape.W, shape.C, generator=torch.Generator().manual_seed(1)).to("cuda", torch.bfloat16)
    return RibLayer(shape, inp, "cuda"), X


def _at_once(jobs):
    """Runs work(failed) of each job in a thread of its own, started together."""
    start, failed = threading.Barrier(len(jobs)), []

    def run(job):
        torch.cuda.set_device(0)
        start.wait()
        try:
            job(failed)
        except Exception as e:   # noqa: BLE001 (told to the main thread)
            failed.append(repr(e))

    threads = [threading.Thread(target=run, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed


def test_projection_and_gate(cuda_lib):
    lib, jobs, checks = cuda_lib.load(), [], []
    for shape in SHAPES + SHAPES:
        lay, X = _layer(shape)
        lay.forward(X)
        torch.cuda.synchronize()
        alone = [t.clone() for t in (lay.Qc, lay.Kc, lay.V, lay.gate)]
        stream = torch.cuda.Stream()
        s, p, f = shape, (lambda t: ctypes.c_void_p(t.data_ptr())), ctypes.c_float
        st = ctypes.c_void_p(stream.cuda_stream)
        # arguments made once: most of a thread's time is spent inside the library, without the interpreter's lock
        qkv = [p(X), 0, s.B, s.H, s.W, s.C, s.heads, s.window, p(lay.Wq), p(lay.Wk), p(lay.Wv), f(1.0 / math.sqrt(lay.dh)), p(lay.Qc),
               p(lay.Kc), p(lay.V), st]
        gate = [p(X), 0, s.B, s.H, s.W, s.C, p(lay.Wdw), p(lay.bdw), p(lay.Wpw), p(lay.bpw), p(lay.gate), None, 0, st]

        def work(failed, qkv=qkv, gate=gate):
            for _ in range(3000):
                if lib.rib_qkv_project(*qkv) or lib.cla_gate(*gate):
                    failed.append(lib.rib_last_error().decode())
                    return

        jobs.append(work)
        checks.append((lay, X, alone, stream))
    _at_once(jobs)
    cuda_lib.rib_device_error()
    for lay, _, alone, _ in checks:
        for a, b in zip(alone, (lay.Qc, lay.Kc, lay.V, lay.gate)):
            assert torch.equal(a, b)


def test_forward_and_backward(cuda_lib):
    jobs, checks = [], []
    for shape in SHAPES + SHAPES:
        lay, X = _layer(shape)
        dY = torch.randn(X.shape, generator=torch.Generator().manual_seed(2)).to("cuda", torch.bfloat16)
        alone = {k: v.clone() for k, v in lay.backward(X, dY).items() if k.startswith("d")}
        stream, out = torch.cuda.Stream(), {}
        torch.cuda.synchronize()

        def work(failed, lay=lay, X=X, dY=dY, stream=stream, out=out):
            with torch.cuda.stream(stream):
                for _ in range(40):
                    out.update(lay.backward(X, dY))
                stream.synchronize()

        jobs.append(work)
        checks.append((alone, out))
    _at_once(jobs)
    cuda_lib.rib_device_error()
    for alone, out in checks:
        for k, v in alone.items():
            assert torch.equal(v, out[k]), k
