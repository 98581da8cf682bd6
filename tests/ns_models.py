"""What a Newton-Schulz result may be off by, sharply: for matrices of many
elements, whose errors' sizes are known and not only bounded."""

import numpy as np

from oracle import step as OS

# A result that misses a remainder, counts it with the wrong sign, or neither.
MISTAKES = {
    "A's diagonal without its remainder": dict(diag_a=0.0),
    "A's remainder subtracted": dict(diag_a=-1.0),
    "B's diagonal without its remainder": dict(diag_b=0.0),
    "B's remainder subtracted": dict(diag_b=-1.0),
    "X without its remainder": dict(rest_x=0.0),
    "X's remainder subtracted": dict(rest_x=-1.0),
}

# at least 15000 elements, and every form of the kernels that one matrix can take
SHAPES = [(60, 250), (250, 60), (128, 192), (192, 128), (40, 700), (700, 40), (120, 700),
          (700, 120), (100, 2500), (2500, 100), (150, 200), (200, 150), (256, 1024), (1024, 256)]


def update(shape, seed, kind):
    """bf16 bits: noise; four directions over noise as strong, or 30 times
    weaker; sixteen directions over noise 300 times weaker."""
    rng = np.random.default_rng(seed)
    k, noise = {"flat": (0, 1.0), "strong": (4, 1.0), "steep": (4, 0.03),
                "sixteen": (16, 0.003)}[kind]
    x = noise * rng.standard_normal(shape)
    if k:
        x = x + rng.standard_normal((shape[0], k)) @ rng.standard_normal((k, shape[1]))
    return OS.f32_to_bf16((1e-3 * x).astype(np.float32))


def rounded(x):
    return OS.bf16_to_f32(OS.f32_to_bf16(np.asarray(x, np.float32))).astype(np.float64)


def off(got, U, steps, coefs):
    """How far `got` is from the iteration in 64 bits, over how far it should
    be.  Two things move it: the output's rounding, by `rnd`, and the binary16
    formats, by |r - e|.  Each entry's rounding to bf16 has little to do with
    what moved the entry before, so their squares add.  The device's binary32
    sums turn a few of the roundings to binary16 around: its errors are others
    than the model's, of the same size.  Both are sums of squares over 15000
    and more entries, which chance leaves within a percent or two of what they
    are expected to be (1/sqrt(15000) = 0.8%, times the entries' unequal
    weights).
    """
    e = OS.newton_schulz(U, steps, coefs)
    r = OS.newton_schulz_rounded(U, steps, coefs)
    rnd = np.linalg.norm(rounded(e) - e)
    return np.linalg.norm(got - e) / np.hypot(rnd, np.linalg.norm(r - e))


ALLOWED = 1.08  # five times that chance


def nearest(got, U, steps, coefs):
    """Which model `got` is nearest to: the one that keeps what the device
    keeps (None), or one with a mistake.  No size of an error enters."""
    full = OS.newton_schulz_rounded(U, steps, coefs)
    best, name = np.linalg.norm(got - full), None
    for what, kw in MISTAKES.items():
        x = OS.newton_schulz_rounded(U, steps, coefs, **kw)
        if not np.array_equal(x, full) and np.linalg.norm(got - x) < best:
            best, name = np.linalg.norm(got - x), what
    return name
