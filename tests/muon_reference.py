"""The Muon step in 64 bits on the host."""
import numpy as np

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orthogonalize(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    a, b, c = coefficients
    x = u / (np.sqrt((u * u).sum()) + eps)
    if x.shape[0] > x.shape[1]:
        return orthogonalize(u.T, steps, coefficients, eps).T
    for _ in range(steps):
        A = x @ x.T
        x = a * x + (b * A + c * (A @ A)) @ x
    return x


def step(p, g, m, lr, momentum, nesterov, weight_decay, scale, grad_scale=1.0, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    """New (p, m, orthogonalised update) of one matrix."""
    g = grad_scale * g
    m = momentum * m + (1 - momentum) * g
    u = (1 - momentum) * g + momentum * m if nesterov else m
    o = orthogonalize(u, steps, coefficients, eps)
    return p * (1 - lr * weight_decay) - lr * scale * o, m, o
