"""Linear attention with one decay per head, and its gradients, in fp64.

    S_t = decay_h S_{t-1} + v_t k_t^T,     o_t = S_t q_t

written out token by token (the definition, and its reverse sweep).  Arrays as in the other
oracles: q, k [B, T, H, d_k], v [B, T, H, d_v], decay [H], states [B, H, d_v, d_k].
"""

import numpy as np


def linear_attention(q, k, v, decay, s0=None):
    """Returns (o, S_T)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    S = np.zeros((B, H, dv, dk)) if s0 is None else s0.astype(np.float64).copy()
    a = np.asarray(decay, dtype=np.float64)[None, :, None, None]
    o = np.empty((B, T, H, dv))
    for t in range(T):
        S = a * S + v[:, t][..., :, None] * k[:, t][..., None, :]
        o[:, t] = np.einsum("bhvk,bhk->bhv", S, q[:, t])
    return o, S


def linear_attention_backward(q, k, v, decay, s0, do, ds_final=None):
    """Returns (dq, dk, dv, ds0) of L = sum <do, o> + <ds_final, S_T>."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    a = np.asarray(decay, dtype=np.float64)[None, :, None, None]
    S = np.zeros((B, H, dv, dk)) if s0 is None else s0.astype(np.float64).copy()
    gq, gk, gv = (np.empty(x.shape) for x in (q, k, v))
    for t in range(T):
        S = a * S + v[:, t][..., :, None] * k[:, t][..., None, :]
        gq[:, t] = np.einsum("bhvk,bhv->bhk", S, do[:, t])
    G = np.zeros((B, H, dv, dk)) if ds_final is None else ds_final.astype(np.float64).copy()
    for t in range(T - 1, -1, -1):
        G = G + do[:, t][..., :, None] * q[:, t][..., None, :]
        gv[:, t] = np.einsum("bhvk,bhk->bhv", G, k[:, t])
        gk[:, t] = np.einsum("bhvk,bhv->bhk", G, v[:, t])
        G = a * G
    return gq, gk, gv, G
