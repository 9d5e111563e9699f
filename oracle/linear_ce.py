"""Softmax cross entropy of z = softcap * tanh(x W^T / softcap) and its gradient
(fp64 oracle; test infrastructure only, see oracle/__init__.py).

Targets outside [0, V) are ignored: loss 0, no gradient.  The mean runs over the
others (0 if there are none).
"""

import numpy as np


def logits(x, w, softcap):
    z = np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
    return softcap * np.tanh(z / softcap) if softcap > 0 else z


def forward(x, w, targets, softcap=0.0):
    """(mean loss, per-token losses [N], log-sum-exp [N])."""
    z = logits(x, w, softcap)
    m = z.max(axis=1)
    lse = m + np.log(np.exp(z - m[:, None]).sum(axis=1))
    valid = (targets >= 0) & (targets < z.shape[1])
    tok = np.where(valid, lse - z[np.arange(len(z)), np.where(valid, targets, 0)], 0.0)
    return (tok[valid].mean() if valid.any() else 0.0), tok, lse


def dlogits(x, w, targets, softcap=0.0, dloss=1.0, dtok=None):
    """dz before the softcap [N, V]: of dloss * mean loss, or of sum dtok * tok_loss."""
    z = logits(x, w, softcap)
    _, _, lse = forward(x, w, targets, softcap)
    valid = (targets >= 0) & (targets < z.shape[1])
    g = np.where(valid, dloss / max(1, valid.sum()) if dtok is None else dtok, 0.0)
    dz = np.exp(z - lse[:, None])
    rows = np.nonzero(valid)[0]
    dz[rows, targets[rows]] -= 1.0
    dz *= g[:, None]
    if softcap > 0:
        dz *= 1.0 - (z / softcap) ** 2
    return dz


def backward(x, w, targets, softcap=0.0, dloss=1.0, dtok=None):
    """(dx [N, d], dW [V, d])."""
    dz = dlogits(x, w, targets, softcap, dloss, dtok)
    return dz @ np.asarray(w, dtype=np.float64), dz.T @ np.asarray(x, dtype=np.float64)
