"""The gated feed-forward projections in float64 (test infrastructure only; page names in
``oracle/__init__.py``).

[Ch. 11.3] and [Paper note] apply LoRA to every linear of the decoder block, its gate and up
projections among them; the block multiplies the activated gate with the up projection:

    [G | L] = X W'^T + LoRA (two linears sharing X),   H = act(G) L
    dG = dH L act'(G),  dL = dH act(G),  then the two linears' gradients

act is x s(z), s the logistic function: z = x (SiLU) or z = 2 sqrt(2/pi) (x + 0.044715 x^3),
which is the tanh form of GELU, since (1 + tanh(z / 2)) / 2 = s(z).
"""

import numpy as np

K2 = 2.0 * np.sqrt(2.0 / np.pi)
CUBIC = 0.044715


def argument(name, x):
    """z and dz/dx."""
    if name == "silu":
        return x, np.ones_like(x)
    return K2 * (x + CUBIC * x ** 3), K2 * (1 + 3 * CUBIC * x ** 2)


def act(name, x):
    """act(x) and act'(x)."""
    z, dz = argument(name, x)
    s = 0.5 * (1 + np.tanh(z / 2))
    small = np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z)))
    s = np.where(z < 0, small, s)
    one_s = np.where(z > 0, small, 1 - s)
    return x * s, s + x * s * one_s * dz


def forward(Y, name):
    G, L = np.split(Y, 2, axis=1)
    return act(name, G)[0] * L


def backward(dH, Y, name):
    """dY = [dG | dL]."""
    G, L = np.split(Y, 2, axis=1)
    f, df = act(name, G)
    return np.concatenate([dH * L * df, dH * f], axis=1)
