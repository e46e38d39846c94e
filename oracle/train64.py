"""fp64 reference of what is trained and scored beside stored layers (CPU,
numpy): low-rank adapters and the vocabulary losses, from their formulas.

TEST INFRASTRUCTURE: shares no code with the HIP path.

  adapters       y_t = W_hat x_t + s_a B_a A_a x_t, a = index[t] in [0, count)
  cross entropy  loss_t = lse(z_t) - z_t[y_t],  z_t = W_hat h_t
  distillation   loss_t = sum_k p_k (log p_k - z_t[i_k] + lse(z_t)),
                 z_t = W_hat h_t / T, p = softmax(teacher / T) over the
                 entries with an index in range and a logit above -inf
"""
from __future__ import annotations

import numpy as np


def adapter_of(index, count):
    """The adapter of each token, -1 for none."""
    index = np.asarray(index, np.int64)
    return np.where((index >= 0) & (index < count), index, -1)


def adapters_forward(x, W_hat, A, B, scaling, index):
    x = np.asarray(x, np.float64)
    y = x @ np.asarray(W_hat, np.float64).T
    for t, a in enumerate(adapter_of(index, len(A))):
        if a >= 0:
            y[t] += scaling[a] * (B[a].astype(np.float64) @ (A[a].astype(np.float64) @ x[t]))
    return y


def adapters_backward(dy, x, W_hat, A, B, scaling, index):
    """(dx, dA, dB) of sum(dy * adapters_forward(x, ...))."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    dx = dy @ np.asarray(W_hat, np.float64)
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    for t, a in enumerate(adapter_of(index, len(A))):
        if a < 0:
            continue
        A64, B64, s = A[a].astype(np.float64), B[a].astype(np.float64), float(scaling[a])
        dv = s * (dy[t] @ B64)
        dx[t] += dv @ A64
        dA[a] += np.outer(dv, x[t])
        dB[a] += s * np.outer(dy[t], A64 @ x[t])
    return dx, dA, dB


def head_targets(index, logits, vocab, temperature=1.0):
    """(m x top entries' probabilities, which take part); labels: logits None."""
    index = np.asarray(index, np.int64)
    if logits is None:
        part = ((index >= 0) & (index < vocab))[:, None]
        return part.astype(np.float64), part
    t = np.asarray(logits, np.float64) / temperature
    part = (index >= 0) & (index < vocab) & (t != -np.inf)
    p = np.zeros(t.shape)
    for i in range(len(t)):
        if part[i].any():
            e = np.exp(t[i, part[i]] - t[i, part[i]].max())
            p[i, part[i]] = e / e.sum()
    return p, part


def head_loss(h, W_hat, index, logits=None, temperature=1.0):
    """(loss, lse, the entries' logits, z)."""
    z = np.asarray(h, np.float64) @ np.asarray(W_hat, np.float64).T / temperature
    top = z.max(1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(1))
    p, part = head_targets(index, logits, z.shape[1], temperature)
    idx = np.asarray(index, np.int64).reshape(len(z), -1)
    loss, zk = np.zeros(len(z)), np.zeros(idx.shape)
    for t in range(len(z)):
        for k in np.nonzero(part[t])[0]:
            zk[t, k] = z[t, idx[t, k]]
            if p[t, k] > 0:
                loss[t] += p[t, k] * (np.log(p[t, k]) - zk[t, k] + lse[t])
    return loss, lse, zk, z


def head_dz(z, index, logits=None, temperature=1.0):
    """d loss / d z: softmax minus what is learnt, 0 for tokens without entries."""
    p, part = head_targets(index, logits, z.shape[1], temperature)
    idx = np.asarray(index, np.int64).reshape(len(z), -1)
    e = np.exp(z - z.max(1, keepdims=True))
    dz = e / e.sum(1, keepdims=True)
    for t in range(len(z)):
        if not part[t].any():
            dz[t] = 0
        for k in np.nonzero(part[t])[0]:
            dz[t, idx[t, k]] -= p[t, k]
    return dz


def head_backward(h, W_hat, index, dloss, logits=None, temperature=1.0):
    z = head_loss(h, W_hat, index, logits, temperature)[3]
    dz = head_dz(z, index, logits, temperature)
    return (np.asarray(dloss, np.float64)[:, None] / temperature) * (dz @ np.asarray(W_hat, np.float64))
