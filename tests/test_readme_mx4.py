"""The README's 4-bit example, run as it is printed (CPU only): the calls stand on the
oracle, the ranks are threads.  No two buffers may be rounded with the same random bits,
and the step has to see the mean over ranks and microbatches."""

import os
import re
import threading
import types

import numpy as np
import pytest

import sharded_bucket_plan_amd as sbp
from oracle import mx4 as OM

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
WORLD, K, LAYERS, STEPS = 3, 2, 2, 2
N = 3 * 96  # a shard: one weight of 3 x 96


def _blocks():
    text = open(README).read()
    text = text[text.index("The exchange in 4-bit floats"):]
    return re.findall(r"```python\n(.*?)```", text, re.S)[:2]


class _Array(np.ndarray):
    """A numpy array that answers to the few torch methods the example uses."""

    def zero_(self):
        self[:] = 0

    def view(self, *shape):
        return self.reshape(shape) if isinstance(shape[0], int) else super().view(*shape)


def _array(x):
    return np.asarray(x, np.float32).view(_Array)


class _Calls:
    """The calls on the oracle; `drawn` holds what names the bits of each random rounding."""

    def __init__(self):
        self.drawn, self.rounded, self.stepped = [], [], None

    def mx_quantize(self, x, along="rows", seed=None, offset=0):
        x = np.asarray(x, np.float32)
        x = x[None] if x.ndim == 1 else x
        if seed is not None:
            assert 0 <= seed < 1 << 64 and 0 <= offset < 1 << 64
            self.drawn.append((seed, offset))

        def value(v, upper):
            code, scale = OM.quantize(v, seed, offset, upper)
            return OM.values(OM.pack(code), scale, v.shape[1]).astype(np.float32)

        made = {"rows": [0], "cols": [1], "both": [0, 1]}[along]
        out = [value(x.T, True) if t else value(x, False) for t in made]
        self.rounded.append(out)
        return tuple(out) if along == "both" else out[0]

    def mx_dequantize(self, q):
        return q

    def mx_reduce_shard(self, peers, acc, scale, out):
        out[:] = OM.reduce([p.reshape(-1) for p in peers], acc, scale)

    def mx_matmul(self, a, b, out=None, accumulate=False):
        c = a.astype(np.float64) @ b.T.astype(np.float64)
        if out is None:
            return c
        out[:] = (out + c if accumulate else c).astype(np.float32)
        return out

    def mean_scale(self, R, micro=1):
        return sbp.mean_scale(R, micro)

    def adamw_shard(self, peers, acc, scale, *rest):
        assert peers == []
        self.stepped = acc * np.float32(scale)


@pytest.fixture(scope="module")
def runs():
    exchange, layer = _blocks()
    rng = np.random.default_rng(1)
    gradients = rng.standard_normal((STEPS, K, WORLD, WORLD, N)).astype(np.float32)
    calls = [[_Calls() for _ in range(WORLD)] for _ in range(STEPS)]
    posts, barrier, failed = [None] * WORLD, threading.Barrier(WORLD), []
    sent_values = np.zeros((STEPS, K, WORLD, WORLD, N), np.float32)

    def one(rank):
        try:
            for step in range(STEPS):
                names = {}

                def all_to_all(sent):
                    for r, q in enumerate(sent):
                        sent_values[step, names["micro"], rank, r] = q[0]
                    posts[rank] = sent
                    barrier.wait(60)
                    got = [posts[r][rank] for r in range(WORLD)]
                    barrier.wait(60)
                    return got

                names.update(
                    sbp=calls[step][rank], world=WORLD, rank=rank, K=K, step=step, layers=LAYERS,
                    rows=3, cols=96, all_to_all=all_to_all, acc=_array(np.full(N, 9.0)),
                    master=_array(rng.standard_normal(N)), m=None, v=None, param_shard=None, hp=None,
                    gradient_chunks=lambda micro: gradients[step, micro, rank])
                exec(exchange, names)
                for micro in range(K):  # the layers' part, in the names that the loop left
                    names["first"] = (micro * WORLD + rank) * (WORLD + LAYERS)
                    for lay in range(LAYERS):
                        local = np.random.default_rng(lay + 10)
                        names.update(layer=lay, x=local.standard_normal((5, 64)),
                                     dy=local.standard_normal((5, 33)),
                                     w=local.standard_normal((33, 64)),
                                     grad=np.zeros((33, 64), np.float32))
                        exec(layer, names)
        except BaseException as e:  # noqa: B902
            failed.append(e)
            barrier.abort()

    threads = [threading.Thread(target=one, args=(r,)) for r in range(WORLD)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    return types.SimpleNamespace(calls=calls, sent=sent_values)


def test_no_two_buffers_are_rounded_with_the_same_bits(runs):
    drawn = [d for of_step in runs.calls for c in of_step for d in c.drawn]
    assert len(drawn) == STEPS * WORLD * K * (WORLD + LAYERS)
    assert len(set(drawn)) == len(drawn)


def test_the_step_sees_the_mean(runs):
    """R * K values an entry, their sum off by one rounding each, and one of the mean."""
    for step in range(STEPS):
        for owner in range(WORLD):
            sent = runs.sent[step][:, :, owner].astype(np.float64).reshape(WORLD * K, N)
            want, size = sent.mean(0), np.abs(sent).mean(0)
            off = np.abs(runs.calls[step][owner].stepped - want)
            assert (off <= (WORLD * K + 2) * 2.0 ** -24 * size).all()
