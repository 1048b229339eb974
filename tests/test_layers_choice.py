"""What a call runs does not depend on the calls before it: sizes, launch limits and
the choice between kernels are the same whichever layer of a process ran first, and
however many host threads make their first calls at once."""

import hashlib
import os
import subprocess
import sys
import threading

import pytest
import torch

from rank_structured_matmul_b200 import layers

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# few rows of long sums: tiles that several CTAs share, more tiles than some
# cluster sizes have clusters
SHAPES = [(16, 1024, 2048), (48, 2048, 2560), (64, 1024, 1536), (100, 1536, 1024),
          (33, 4096, 1024), (128, 2048, 2048), (201, 1280, 5120)]


def case(N, d_in, d_out, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + N + d_in + d_out)
    X = torch.randn(N, d_in, generator=g, device="cuda").bfloat16()
    W = (torch.randn(d_out, d_in, generator=g, device="cuda") * d_in ** -0.5).bfloat16()
    return X, W


def bits(N, d_in, d_out):
    layer = layers.DenseLinear(d_in, d_out)
    X, W = case(N, d_in, d_out)
    Y = layer.forward(X, W)
    dX, dW, db = layer.backward(Y, X, W)
    assert layer.status() == 0
    layer.close()
    h = hashlib.sha256()
    for t in (Y, dX, dW, db):
        h.update(t.cpu().view(torch.int16).numpy().tobytes())
    return h.hexdigest()[:16]


def in_a_fresh_process(first):
    code = ("import sys; sys.path.insert(0, %r); sys.path.insert(0, %r)\n"
            "import test_layers_choice as t\n"
            "for s in %r: t.bits(*s)\n"
            "print('bits', *[t.bits(*s) for s in t.SHAPES])\n"
            % (ROOT, os.path.join(ROOT, "tests"), first))
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                         timeout=600)
    assert out.returncode == 0, out.stderr[-3000:]
    return [line for line in out.stdout.splitlines() if line.startswith("bits")][-1]


@pytest.mark.parametrize("first", [[(16, 128, 64)], [(16, 64, 2048), (128, 256, 128)]])
def test_bits_do_not_depend_on_the_first_call(first):
    assert in_a_fresh_process(first) == in_a_fresh_process([])


def test_first_calls_from_many_threads():
    """Handles of their own, a stream each: every call succeeds, in the bits of the
    same call alone."""
    sizes = [(n, d, 264) for n in (1, 17, 40, 70, 100, 127, 300) for d in (136, 520)]
    got, errors = {}, []

    def work(s):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                layer = layers.DenseLinear(*s[1:])
                X, W = case(*s)
                Y = layer.forward(X, W, act="gelu")
                stream.synchronize()
                got[s] = Y
                assert layer.status() == 0
                layer.close()
        except Exception as e:  # reported below, in the main thread
            errors.append((s, e))

    threads = [threading.Thread(target=work, args=(s,)) for s in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for s in sizes:
        layer = layers.DenseLinear(*s[1:])
        X, W = case(*s)
        assert torch.equal(got[s], layer.forward(X, W, act="gelu"))
        layer.close()
