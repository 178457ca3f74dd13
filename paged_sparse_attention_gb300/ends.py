"""The two ends of a model around its layers, chunk by chunk, through the C ABI.

In front: the embeddings of the tokens (oomb_embed_fwd).  Behind: the last layer norm
(oomb_layer_norm_fwd), where the model has one, and softmax cross entropy over the vocabulary
(oomb_head_loss_fwd), whose logits are never kept: chunk-recurrent training ("Out of the Memory
Barrier", gist.science explainer, 2.A) holds the activations of one chunk, and the logits of one
chunk of 8192 tokens over 131072 entries would be 4.3 GB.  The loss of a chunk and its gradients are
formed together, where the reverse sweep has the chunk's last hidden states at hand: ``behind``
returns what LayerStep.run takes in place of dO.

This module only orders calls.  Gradients are summed in fp32 over the chunks: of the table (by
sorted tokens, oomb_embed_bwd), of the output projection, of the norm's parameters.
"""
from __future__ import annotations

import torch

from . import _lib as L


class ModelEnds:
    """``table`` [V, Dm] (bf16 or fp32, device): the embeddings.  ``head`` [V, Dm] (the same dtype): the
    output projection, with a gradient of its own; None: the table itself, whose gradient then holds both
    shares.  ``w_norm``, ``b_norm`` (fp32 [Dm] or None): the last layer norm, there when ``w_norm`` is.  ``scale``: factor of
    the embeddings; ``softcap``: cap of the logits (0: none).  ``chunk``: most tokens of a call.

    Gradients, zeroed by ``zero_grad``: d_table, d_head (the same tensor when shared), and dw_norm,
    db_norm where the norm has them, all fp32.  Calls of one object follow one another on one stream: they share a
    workspace and the gradients.  Errors that kernels met (a token behind the vocabulary)
    are told by ``check``."""

    def __init__(self, table, head=None, w_norm=None, b_norm=None, chunk: int = 4096, scale: float = 1.0,
                 softcap: float = 0.0, eps: float = 1e-5):
        if table.dim() != 2 or (head is not None and (head.shape != table.shape or head.dtype != table.dtype)):
            raise ValueError("ModelEnds: table and head are [V, Dm] of one dtype")
        if w_norm is None and b_norm is not None:
            raise ValueError("ModelEnds: b_norm belongs to the norm (w_norm)")
        if chunk < 1:
            raise ValueError("ModelEnds: chunk has to be positive")
        self.table, self.head = table, table if head is None else head
        self.w_norm, self.b_norm, self.chunk = w_norm, b_norm, chunk
        self.scale, self.softcap, self.eps = scale, softcap, eps
        self.V, self.Dm = table.shape
        self.dev, self.dtype = table.device, table.dtype
        f32 = dict(dtype=torch.float32, device=self.dev)
        self.d_table = torch.zeros((self.V, self.Dm), **f32)
        self.d_head = self.d_table if head is None else torch.zeros((self.V, self.Dm), **f32)
        self.dw_norm = None if w_norm is None else torch.zeros(self.Dm, **f32)
        self.db_norm = None if b_norm is None else torch.zeros(self.Dm, **f32)
        self.word = torch.zeros(1, dtype=torch.int32, device=self.dev)
        # calls of both ends come one after another on a stream: one workspace serves them all
        size = max(L.oomb_embed_workspace(chunk, self.Dm),
                   L.oomb_head_loss_workspace(chunk, self.Dm, self.V, self.dtype, True),
                   0 if w_norm is None else L.oomb_layer_norm_workspace(chunk, self.Dm))
        self.ws = torch.empty(size, dtype=torch.uint8, device=self.dev)

    def zero_grad(self) -> None:
        for g in (self.d_table, self.d_head, self.dw_norm, self.db_norm):
            if g is not None:
                g.zero_()

    def embed(self, tokens):
        """X [N, Dm] of tokens int64 [N] (a negative one is none: zeros)."""
        X = torch.empty((tokens.shape[0], self.Dm), dtype=self.dtype, device=self.dev)
        L.oomb_embed_fwd(tokens, self.table, X, self.word, scale=self.scale)
        return X

    def embed_grad(self, tokens, dX) -> None:
        """Adds to d_table from the gradient dX [N, Dm] (bf16 or fp32) of ``embed``'s result."""
        for s in range(0, tokens.shape[0], self.chunk):
            L.oomb_embed_bwd(tokens[s:s + self.chunk], dX[s:s + self.chunk], self.d_table, self.ws, self.word,
                             scale=self.scale, accumulate=True)

    def chunk_loss(self, h, targets, loss, weights=None, scale: float = 1.0, grads: bool = True):
        """``loss`` [n] (fp32, written) of the hidden states h [n, Dm] of one chunk, targets int64 [n] (a
        negative one is none).  With ``grads`` also dh, the gradient of scale * sum(weights * loss), its
        share of the parameters' added to theirs."""
        n = h.shape[0]
        if n > self.chunk:
            raise ValueError(f"ModelEnds: a chunk of {n} tokens, at most {self.chunk}")
        f32 = dict(dtype=torch.float32, device=self.dev)
        u = h
        if self.w_norm is not None:
            mean, rstd = (torch.empty(n, **f32) if grads else None for _ in range(2))
            u = torch.empty_like(h)
            L.oomb_layer_norm_fwd(h, self.w_norm, self.b_norm, u, eps=self.eps, mean=mean, rstd=rstd)
        lse = torch.empty(n, **f32)
        L.oomb_head_loss_fwd(u, self.head, targets, loss, lse, self.ws, self.word, softcap=self.softcap)
        if not grads:
            return None
        du = torch.empty_like(u)
        L.oomb_head_loss_bwd(u, self.head, targets, lse, du, self.d_head, self.ws, self.word, d_loss=weights, scale=scale,
                             softcap=self.softcap, accumulate=True)
        if self.w_norm is None:
            return du
        dh = torch.empty_like(h)
        L.oomb_layer_norm_bwd(h, self.w_norm, mean, rstd, du, dh, dw=self.dw_norm, db=self.db_norm, accumulate=True,
                              workspace=self.ws)
        return dh

    def behind(self, targets, loss, weights=None, scale: float = 1.0):
        """What LayerStep.run takes in place of dO: called with a chunk's first token and its attention
        output o [n, Hq, d] (Hq d = Dm), it writes the chunk's share of ``loss`` [N] (fp32) and returns the
        gradient of scale * sum(weights * loss).  targets int64 [N]; weights fp32 [N] or None."""

        def d_o(start: int, o):
            n = o.shape[0]
            cut = slice(start, start + n)
            dh = self.chunk_loss(o.view(n, self.Dm), targets[cut], loss[cut], None if weights is None else weights[cut],
                                 scale)
            return dh.view_as(o)

        return d_o

    def check(self) -> None:
        """Raises OombError if a kernel has met an error since the last check (synchronizes)."""
        L.oomb_word_check(self.word)
