"""The MLP half of a pre-norm transformer block on the Lynx layer.

    X  = layer_norm(h)
    H  = gelu(S(X) Wu^T + bu + (X Au^T) Bu^T)
    h' = h + S(H) Wd^T + bd + (H Ad^T) Bd^T

W frozen, the adapters, the biases and the norm trained.  The norm and the two
layers with GELU and the residual stream in their epilogues are one call of the
library each, and so are for a training step the 8-bit checkpoints of X and H, the
selections the forward pass made and Z, from which ``backward`` takes every
gradient (torch copies a selection out of its workspace, and transposes the adapter
of a layer that selective skipping leaves dense).  ``forward_few`` serves up to 32
tokens on the weights in 4 bits.

Everything runs on the current stream, captured or not.  Nothing is kept from one
step for the next but the layouts of W (W^T from the first backward pass that is not
captured: a graph captured before it transposes W in every replay).
"""
from . import lynx


class MlpBlock:
    """``up`` and ``down`` are dicts with CUDA bf16 tensors ``W`` [N,K], ``bias`` [N]
    or None, ``A`` [r,K] and ``B`` [N,r] (or both None), and ``skip``: True for a layer
    that selective skipping leaves dense.  ``norm`` is (weight, bias), each [K] or None.
    Both widths are multiples of 64 (the backward pass sums over them)."""

    def __init__(self, norm, up, down, eps=1e-6, checkpoint=lynx.LYNX_CKPT8_INT8):
        self.weight, self.bias = norm
        self.up, self.down = dict(up), dict(down)
        self.eps = float(eps)
        self.checkpoint = checkpoint
        if self.up["W"].shape != self.down["W"].shape[::-1]:
            raise ValueError("down must lead back from up's width")
        for layer in (self.up, self.down):
            N, K = layer["W"].shape
            if N % 64 or K % 64:
                raise ValueError("both widths must be multiples of 64")
            layer.setdefault("skip", False)
            layer["Wt"] = None  # W^T, laid out once before the first backward pass
            layer["w4"] = None

    def _layer(self, layer, X, keep, **kw):
        """One layer's Y and Z, and what its backward pass needs."""
        import torch

        ws = None
        if keep and not layer["skip"]:  # the selection is taken from it
            r = layer["A"].shape[0] if layer["A"] is not None else 0
            ws = torch.empty(lynx.lynx_workspace_bytes(X.shape[0], *layer["W"].shape, r), dtype=torch.uint8,
                             device=X.device)
        Y, Z = lynx.lynx_linear_residual(X, layer["W"], layer["bias"], layer["A"], layer["B"],
                                         skip_sparsify=layer["skip"], workspace=ws, **kw)
        if not keep:
            return Y, None
        meta = None if layer["skip"] else lynx.lynx_workspace_meta(ws, *X.shape).clone()
        return Y, (*lynx.lynx_ckpt8_store(X, format=self.checkpoint), meta, Z)

    def forward(self, h, train=False):
        """h' [M,K]; with ``train`` (h', saved), ``saved`` for ``backward``: it holds h itself, which
        must stay as it is until then."""
        if not train:
            X = lynx.lynx_layer_norm(h, self.weight, self.bias, eps=self.eps)
            H, _ = self._layer(self.up, X, False, act=lynx.LYNX_ACT_GELU_TANH)
            return self._layer(self.down, H, False, R=h)[0]
        X, mean, rstd = lynx.lynx_layer_norm(h, self.weight, self.bias, eps=self.eps, want_stats=True)
        H, up = self._layer(self.up, X, True, act=lynx.LYNX_ACT_GELU_TANH, want_Z=True)
        out, down = self._layer(self.down, H, True, R=h)
        return out, (h, mean, rstd, up, down)

    @staticmethod
    def _transposed(layer):
        import torch

        if layer["Wt"] is not None:
            return layer["Wt"]
        Wt = layer["W"].t().contiguous()
        if not torch.cuda.is_current_stream_capturing():  # a capture's is the graph's, filled when it is replayed
            torch.cuda.current_stream().synchronize()  # once: later steps may be on other streams
            layer["Wt"] = Wt
        return Wt

    @classmethod
    def _layer_backward(cls, layer, dP, q, e, meta, want):
        """dX of one layer from the gradient of P, and the adapter's gradients into ``want``."""
        Wt = cls._transposed(layer)
        A, B = layer["A"], layer["B"]
        dT = None
        if A is not None:
            want["A"], want["B"], dT = lynx.lynx_lora_backward(dP, q, e, A, B)
        if layer["skip"]:
            if A is None:
                return lynx.lynx_linear_dense(dP, Wt)
            return lynx.lynx_linear_dense(dP, Wt, None, B.t().contiguous(), A.t().contiguous())
        G = lynx.lynx_linear_dense(dP, Wt)
        return lynx.lynx_sparsify_backward(G, q, e, dT, A, meta=meta)

    def backward(self, saved, dout):
        """(dh, gradients) from the gradient of h'.  ``gradients`` has "norm": (dweight,
        dbias), and "up" and "down": dicts with "bias", "A" and "B" where the layer has them.
        The gradients of a parameter that is None are None or left out."""
        h, mean, rstd, (qx, ex, mx, Z), (qh, eh, mh, _) = saved
        up, down = {}, {}
        if self.down["bias"] is not None:
            _, down["bias"] = lynx.lynx_act_backward(dout, act=lynx.LYNX_ACT_NONE)
        dH = self._layer_backward(self.down, dout, qh, eh, mh, down)
        dZ, dbias = lynx.lynx_act_backward(dH, Z, want_bias=self.up["bias"] is not None, dZ=dH)
        if dbias is not None:
            up["bias"] = dbias
        dX = self._layer_backward(self.up, dZ, qx, ex, mx, up)
        dh, dweight, dnorm = lynx.lynx_layer_norm_backward(dX, h, mean, rstd, self.weight, dR=dout,
                                                           want_weight=self.weight is not None,
                                                           want_bias=self.bias is not None)
        return dh, {"norm": (dweight, dnorm), "up": up, "down": down}

    def quantize(self, group=128, zero_points=True):
        """Lay out the weights in 4 bits for ``forward_few`` (the bf16 weights stay).  Waits
        for the current stream: ``forward_few`` may follow on any.  Not inside a capture.
        Laid out again, the layout before is given up: graphs captured on it are void."""
        import torch

        if torch.cuda.is_current_stream_capturing():  # the graph's memory, without values until it is replayed
            raise RuntimeError("quantize() before the capture")
        laid = [lynx.lynx_w4_quantize(layer["W"], group, zero_points=zero_points) for layer in (self.up, self.down)]
        torch.cuda.current_stream().synchronize()
        self.up["w4"], self.down["w4"] = laid

    def forward_few(self, h):
        """h' for up to 32 tokens on the weights in 4 bits (``quantize`` first), both
        layers dense."""
        if self.up["w4"] is None:
            raise RuntimeError("quantize() first")
        X = lynx.lynx_layer_norm(h, self.weight, self.bias, eps=self.eps)
        H = lynx.lynx_linear_w4(X, *self.up["w4"], self.up["bias"], self.up["A"], self.up["B"],
                                act=lynx.LYNX_ACT_GELU_TANH)
        return lynx.lynx_linear_w4_residual(H, *self.down["w4"], self.down["bias"], self.down["A"], self.down["B"], R=h)
