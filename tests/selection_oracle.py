"""The gradient through S(X) with a given selection, in 64 bits."""
import torch

import adapter_oracle as ao
import helpers


def from_metadata(meta, M, K):
    """m [M,K] (0 or 1, float64) from hardware metadata bytes on any device."""
    canon = torch.from_numpy(helpers.canonical_from_hw(meta.cpu().numpy(), M, K).copy()).to(meta.device)
    nib = torch.stack([canon & 15, canon >> 4], dim=2).reshape(M, K // 4).long()
    at = torch.arange(4, device=meta.device)
    m = (at == (nib & 3)[..., None]) | (at == (nib >> 2)[..., None])
    return m.reshape(M, K).double()


def layer(x, m):
    """S(x) = s m x with the selection m fixed."""
    L, Lk = x.abs().sum(1, keepdim=True), (m * x.abs()).sum(1, keepdim=True)
    return torch.where(Lk > 0, L / torch.where(Lk > 0, Lk, 1.0), 1.0) * m * x


def gradient(G, x, m, dT=None, A=None):
    """(dX, bound on |error|) at x with the selection m; the bound as in adapter_oracle."""
    G = G.double()
    K = x.shape[1]
    L, Lk = x.abs().sum(1, keepdim=True), (m * x.abs()).sum(1, keepdim=True)
    some = Lk > 0
    safe = torch.where(some, Lk, 1.0)
    s = torch.where(some, L / safe, 1.0)
    D = (m * G * x).sum(1, keepdim=True)
    dX = s * m * G + torch.where(some, torch.sign(x) * (D / safe) * (1 - s * m), 0.0)
    size = s * m * G.abs() + (m * (G * x).abs()).sum(1, keepdim=True) / safe * (1 + s * m)
    tol = 2 * (K + 16) * ao.F32 * size
    if dT is not None:
        dT, A = dT.double(), A.double()
        dX = dX + dT @ A
        tol = tol + (A.shape[0] + 16) * ao.F32 * (dT.abs() @ A.abs())
    return dX, 1.01 * (ao.BF * dX.abs() + tol) + ao.TINY
