"""One attention layer of a decode step around the library's attention: of one token a sequence (``DecodeLayer``),
or of a drafted tree of tokens whose accepted path is committed afterwards (``TreeLayer``).

What a layer does with the step's hidden vectors, in the order of its calls:

    q    = Wq x                       csa2_linear_fp4, all heads at once
    q, k = norm and rotation          csa2_norm_rope: the query heads in place, the token's own
                                      latent row into its slot of the window
    o    = attention                  csa2_sparse_attn over given indices (with their window), or
                                      csa2_dense_attn over every visible entry
    o    = rotated back               csa2_norm_rope by the query's position, fp32 or bf16 -> bf16:
                                      the latent is the value too, so its rotated part comes out
                                      turned by the keys' positions
    y    = Wo o, head group by group  csa2_linear_fp4

"DeepSeek-v4.1 Flash: KVキャッシュ圧縮の限界を押し広げる" §1.2 names the low-rank query projection, the
rotated part of the latent and the grouped output projection; the pages give no weights, so the
caller's are used, held in the cache's FP4 format.
"""
import torch

from . import (D_LAT, EVERY_ENTRY, OP_DENSE_ATTN, OP_LINEAR_FP4, OP_SPARSE_ATTN, OP_TREE_ATTN, WINDOW_AT_QUERY,
               csa2_cache_append, csa2_dense_attn, csa2_linear_fp4, csa2_norm_rope, csa2_quantize_fp4, csa2_sparse_attn,
               csa2_tree_attn, workspace)
from .decode import _Graphed


def quantize_weight(w):
    """an fp32 matrix [.., n_out, n_in] as (codes, scales, alpha): values times 1/alpha in FP4, alpha the
    power of two that puts the largest magnitude into [3 * 2^7, 3 * 2^8), so that the E4M3 scales of its groups
    (a sixth of the group's largest value) lie at the top of their range and small ones stay normal"""
    top = float(w.abs().max())
    e = 0 if top == 0 or not torch.isfinite(torch.tensor(top)) else 8 - int(torch.frexp(torch.tensor(top / 3.0))[1])
    codes, scales = csa2_quantize_fp4((w.float() * 2.0 ** e).contiguous())
    return codes, scales, 2.0 ** -e


class DecodeLayer(_Graphed):
    """Buffers and calls of one layer for B sequences, one token each.

    wq fp32 [H * 512, r_q]; wo fp32 [groups, r_out, (H / groups) * 512]; q_weight, k_weight fp32 [512]
    (the norms' weights); rot: how many of the last values are rotated, with frequencies
    base^(-2i/rot).  The caller fills x [B, r_q] and row [B, 512] (the token's latent row) and pos
    [B], keeps the earlier tokens' rows in win [B, 128, 512] (oldest first; the last is this
    token's, written by the step, so that the first is of position pos - 127), and runs enqueue()
    (or capture() once and run()).  With idx int32 [B, 1, k] the attention reads those entries,
    else every visible one.  The window lies where pos puts it, at every step and in a graph too
    (swa_pos0 is taken for callers that pass it and not used).  The result is y [B, groups, r_out]."""

    def __init__(self, cache, wq, wo, q_weight, k_weight, rot=64, base=10000.0, eps=1e-6, idx=None, swa_pos0=None,
                 out_dtype=torch.bfloat16):
        dev, B = cache.lat_codes.device, cache.batch
        bf16 = torch.bfloat16
        self.cache, self.idx, self.eps, self.B = cache, idx, eps, B
        self.H = wq.shape[0] // D_LAT
        self.groups, r_out = wo.shape[0], wo.shape[1]
        self.wq, self.wo = quantize_weight(wq), quantize_weight(wo)
        self.q_weight, self.k_weight = q_weight, k_weight
        self.inv_freq = (float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(dev)
        # inputs
        self.x = torch.zeros((B, wq.shape[1]), dtype=bf16, device=dev)
        self.row = torch.zeros((B, 1, D_LAT), dtype=bf16, device=dev)
        self.pos = torch.zeros((B,), dtype=torch.int64, device=dev)
        self.win = torch.zeros((B, 128, D_LAT), dtype=bf16, device=dev)
        # without idx: the position of each window's first row, set by the step
        self.win_pos0 = torch.zeros((B,), dtype=torch.int64, device=dev)
        # intermediates and the result
        self.q = torch.empty((B, self.H, D_LAT), dtype=bf16, device=dev)
        self.o = torch.empty((B, 1, self.H, D_LAT), dtype=bf16 if idx is None else torch.float32, device=dev)
        self.o16 = torch.empty((B, self.H, D_LAT), dtype=bf16, device=dev)
        self.y = torch.empty((B, self.groups, r_out), dtype=out_dtype, device=dev)
        k = 0 if idx is None else idx.shape[-1]
        self.ws = workspace(OP_DENSE_ATTN if idx is None else OP_SPARSE_ATTN, B, 1, self.H, k, cache.capacity, dev)
        self.ws_q = workspace(OP_LINEAR_FP4, B, 1, 0, 0, wq.shape[1], dev)
        self.ws_o = workspace(OP_LINEAR_FP4, B, self.groups, 0, 0, wo.shape[2], dev)

    def enqueue(self, stream=None):
        if self.idx is None:
            with torch.cuda.stream(stream):      # (None: the current one)
                torch.sub(self.pos, self.win.shape[1] - 1, out=self.win_pos0)
        codes, scales, alpha = self.wq
        csa2_linear_fp4(self.x, codes, scales, alpha, out=self.q.view(self.B, -1), ws=self.ws_q, stream=stream)
        csa2_norm_rope(self.q, self.pos, self.inv_freq, q_weight=self.q_weight, k=self.row, k_weight=self.k_weight,
                       eps=self.eps, q_out=self.q, k_out=self.win[:, -1:], stream=stream)
        q, q_pos = self.q.view(self.B, 1, self.H, D_LAT), self.pos.view(self.B, 1)
        if self.idx is None:
            csa2_dense_attn(self.cache, q, q_pos, self.win, self.win_pos0, out=self.o, ws=self.ws, stream=stream)
        else:
            csa2_sparse_attn(self.cache, q, q_pos, self.idx, self.win, WINDOW_AT_QUERY, out=self.o, ws=self.ws,
                             stream=stream)
        csa2_norm_rope(self.o.view(self.B, self.H, D_LAT), self.pos, self.inv_freq, norm=False, inverse=True,
                       q_out=self.o16, stream=stream)
        codes, scales, alpha = self.wo
        csa2_linear_fp4(self.o16.view(self.B, self.groups, -1), codes, scales, alpha, out=self.y, ws=self.ws_o,
                        stream=stream)


class TreeLayer(_Graphed):
    """Buffers and calls of one layer for B drafted trees of up to `nodes` tokens (at most 128).

    Weights, rot, base and eps as in DecodeLayer.  The caller fills x [B, n, r_q], row [B, n, 512] (the nodes'
    latent rows), parent [B, n] (an earlier node, -1: a child of the last committed token, -2: not there) and pos
    [B, n] (raw positions), keeps the committed rows in win [B, 128, 512] (the last is of position
    committed[b] - 1, oldest first), and runs enqueue() (or capture() once and run()).  With idx int32 [B, n, k]
    a node reads the entries of its list, else every visible one.  The attention's outputs are held in bf16 with
    and without lists, with weights of 2^-11 (DecodeLayer's in fp32 with idx: one rounding of 2^-8 less before Wo; for a
    tree of 16 nodes over 512 entries fp32 would take 70 us where bf16 takes 56).  The result is y [B, n, groups, r_out];
    rows of nodes that are not there hold nothing of use.  commit() then takes an accepted path over."""

    def __init__(self, cache, wq, wo, q_weight, k_weight, nodes, rot=64, base=10000.0, eps=1e-6, idx=None,
                 out_dtype=torch.bfloat16):
        dev, B, n = cache.lat_codes.device, cache.batch, nodes
        bf16 = torch.bfloat16
        self.cache, self.idx, self.eps, self.B, self.n = cache, idx, eps, B, n
        self.H = wq.shape[0] // D_LAT
        self.groups, r_out = wo.shape[0], wo.shape[1]
        self.wq, self.wo = quantize_weight(wq), quantize_weight(wo)
        self.q_weight, self.k_weight = q_weight, k_weight
        self.inv_freq = (float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(dev)
        # inputs
        self.x = torch.zeros((B, n, wq.shape[1]), dtype=bf16, device=dev)
        self.row = torch.zeros((B, n, D_LAT), dtype=bf16, device=dev)
        self.parent = torch.full((B, n), -2, dtype=torch.int32, device=dev)
        self.pos = torch.zeros((B, n), dtype=torch.int64, device=dev)
        self.win = torch.zeros((B, 128, D_LAT), dtype=bf16, device=dev)
        self.committed = torch.zeros((B,), dtype=torch.int64, device=dev)
        # intermediates and the result
        self.win_pos0 = torch.zeros((B,), dtype=torch.int64, device=dev)
        self.draft = torch.empty((B, n, D_LAT), dtype=bf16, device=dev)
        self.q = torch.empty((B, n, self.H, D_LAT), dtype=bf16, device=dev)
        self.o = torch.empty((B, n, self.H, D_LAT), dtype=bf16, device=dev)
        self.y = torch.empty((B, n, self.groups, r_out), dtype=out_dtype, device=dev)
        k = EVERY_ENTRY if idx is None else idx.shape[-1]
        self.ws = workspace(OP_TREE_ATTN, B, n, self.H, k, cache.capacity, dev)
        self.ws_q = workspace(OP_LINEAR_FP4, B * n, 1, 0, 0, wq.shape[1], dev)
        self.ws_o = workspace(OP_LINEAR_FP4, B * n, self.groups, 0, 0, wo.shape[2], dev)

    def enqueue(self, stream=None):
        T, H = self.B * self.n, self.H
        with torch.cuda.stream(stream):          # (None: the current one)
            torch.sub(self.committed, self.win.shape[1], out=self.win_pos0)
        codes, scales, alpha = self.wq
        csa2_linear_fp4(self.x.view(T, -1), codes, scales, alpha, out=self.q.view(T, -1), ws=self.ws_q, stream=stream)
        q, pos = self.q.view(T, H, D_LAT), self.pos.view(T)
        csa2_norm_rope(q, pos, self.inv_freq, q_weight=self.q_weight, k=self.row.view(T, 1, D_LAT), k_weight=self.k_weight,
                       eps=self.eps, q_out=q, k_out=self.draft.view(T, 1, D_LAT), stream=stream)
        csa2_tree_attn(self.cache, self.q, self.pos, self.parent, self.draft, self.win, self.win_pos0, idx=self.idx,
                       out=self.o, ws=self.ws, stream=stream)
        o = self.o.view(T, H, D_LAT)
        csa2_norm_rope(o, pos, self.inv_freq, norm=False, inverse=True, q_out=o, stream=stream)
        codes, scales, alpha = self.wo
        csa2_linear_fp4(self.o.view(T, self.groups, -1), codes, scales, alpha, out=self.y.view(T, self.groups, -1),
                        ws=self.ws_o, stream=stream)

    def commit(self, path, h=None, prev=None, w0=None, w1=None, wik_codes=None, wik_scales=None, stream=None):
        """the accepted path int32 [B, m] (node numbers from the root's child on, ended by its first that is no
        node): its draft rows move into the window, and the committed positions on.  With h bf16 [B, n, 512], the
        nodes' rows that the cache is made of, they are appended to it too (prev, w0, w1 and the projection as in
        csa2_cache_append; prev is carried on in place): once for the layers that share a cache.  It reads what
        enqueue() wrote and changes what the next one reads: on the same stream, or behind it."""
        with torch.cuda.stream(stream):          # (None: the current one)
            if h is not None:
                csa2_cache_append(self.cache, h, self.committed, path=path, prev=prev, prev_out=prev, w0=w0, w1=w1,
                                  wik_codes=wik_codes, wik_scales=wik_scales, stream=stream)
            length = ((path >= 0) & (path < self.n)).long().cumprod(1).sum(1)
            at = path.long().clamp(0, self.n - 1)[..., None].expand(-1, -1, D_LAT)
            rows = torch.cat((self.win, self.draft.gather(1, at)), 1)
            keep = torch.arange(128, device=path.device) + length[:, None]
            self.win.copy_(rows.gather(1, keep[..., None].expand(-1, -1, D_LAT)))
            self.committed += length
