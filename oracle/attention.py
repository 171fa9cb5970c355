"""fp64 CPU definitions of linear attention with a decay per head and of paged decode
attention.  Test infrastructure only; shares no code with the CUDA path.

Plain token loops of the definitions

    S_t = a S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t          (a = exp(log_decay))
    o = softmax(scale q K^T) V     over the keys of a row's pages

on the exact input values.  The gradients walk the adjoint recurrence
D_t = scale q_t do_t^T + a D_{t+1}; a test holds them against torch.autograd of the forward
loop and against differences.
"""
from __future__ import annotations

import math

import torch


def _f64(x):
    return None if x is None else x.detach().cpu().double()


def _decay(log_decay):
    return 1.0 if log_decay is None else torch.exp(_f64(log_decay))[:, None, None]


def la_forward(q, k, v, log_decay, initial_state=None, scale=None):
    """(out [B,T,H,dv], final_state [B,H,dk,dv]) as fp64 tensors; differentiable in fp64 inputs."""
    cast = (lambda x: x) if q.dtype == torch.float64 else _f64
    q, k, v = cast(q), cast(k), cast(v)
    B, T, H, dk = q.shape
    scale = 1.0 / math.sqrt(dk) if scale is None else scale
    a = _decay(log_decay)
    S = torch.zeros((B, H, dk, v.shape[-1]), dtype=torch.float64)
    if initial_state is not None:
        S = initial_state if initial_state.dtype == torch.float64 else _f64(initial_state)
    out = []
    for t in range(T):
        S = a * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        out.append(scale * torch.einsum("bhc,bhcd->bhd", q[:, t], S))
    return (torch.stack(out, 1) if out else v.new_zeros(v.shape)), S


def la_backward(q, k, v, log_decay, grad_out, initial_state=None, grad_final_state=None, scale=None):
    """dict dq, dk, dv, dinitial_state (fp64) of la_forward."""
    q, k, v, do = _f64(q), _f64(k), _f64(v), _f64(grad_out)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    scale = 1.0 / math.sqrt(dk) if scale is None else scale
    a = _decay(log_decay)
    S = torch.zeros((B, H, dk, dv), dtype=torch.float64) if initial_state is None else _f64(initial_state)
    D = torch.zeros((B, H, dk, dv), dtype=torch.float64) if grad_final_state is None else _f64(grad_final_state)
    g = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v))
    for t in range(T):
        S = a * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        g["dq"][:, t] = scale * torch.einsum("bhcd,bhd->bhc", S, do[:, t])
    for t in reversed(range(T)):
        D = D + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        g["dk"][:, t] = torch.einsum("bhcd,bhd->bhc", D, v[:, t])
        g["dv"][:, t] = torch.einsum("bhcd,bhc->bhd", D, k[:, t])
        D = a * D
    g["dinitial_state"] = D
    return g


def paged_decode(q, k, v, k_cache, v_cache, block_table, lengths, scale=None):
    """(out, magnitude, k_cache, v_cache): the outputs and sum_j p_j |v_j| in fp64 (None rows of
    idle sequences are NaN), and the caches with the new keys and values in their own dtype."""
    q64, table, kc, vc = _f64(q), block_table.cpu().long(), k_cache.cpu().clone(), v_cache.cpu().clone()
    B, H, D = q64.shape
    num_pages, page, Hkv = kc.shape[:3]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    rows = [int(n) for n in lengths.cpu()]
    keys = [-1 if n < 0 or n + (k is not None) > table.shape[1] * page else n + (k is not None) for n in rows]
    inside = lambda p: 0 <= p < num_pages
    if k is not None:
        for b, n in enumerate(rows):
            if keys[b] > 0 and inside(int(table[b, n // page])):
                kc[table[b, n // page], n % page], vc[table[b, n // page], n % page] = k[b].cpu(), v[b].cpu()
    out = torch.full((B, H, D), math.nan, dtype=torch.float64)
    mag = torch.full((B, H, D), math.nan, dtype=torch.float64)
    group = H // Hkv
    for b, n in enumerate(keys):
        if n < 0:
            continue
        at = torch.arange(n)
        pages = table[b, at // page] if n else at
        own = (at == rows[b]) if k is not None else torch.zeros(n, dtype=torch.bool)
        good = (pages >= 0) & (pages < num_pages)
        kk, vv = kc[pages.clamp(0, num_pages - 1), at % page].double(), vc[pages.clamp(0, num_pages - 1), at % page].double()
        if k is not None and n:
            kk[own], vv[own] = k[b].cpu().double(), v[b].cpu().double()
        kk, vv = kk[good | own], vv[good | own]
        for h in range(H):
            x = scale * (kk[:, h // group] @ q64[b, h])
            p = torch.softmax(x, 0) if x.numel() else x
            out[b, h] = p @ vv[:, h // group]
            mag[b, h] = p @ vv[:, h // group].abs()
    return out, mag, kc, vc
