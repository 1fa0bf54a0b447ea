"""Verify-step executor: a fixed sequence of libw12 calls over preallocated
device buffers, captured once into a CUDA graph and replayed per step.

A verify step at batch B x block T runs each target linear (W12 GEMM) on its
activation rows and finishes with the fused W12 LM head, row argmax and
greedy acceptance. The layer's GEMMs, whose inputs are all given, run as one
grouped launch (w12_gemm_grouped: one persistent kernel, one ramp-up and one
tail for all of them) unless grouped=False asks for one launch per GEMM.
Capturing the launches removes per-call host overhead (Python, ctypes,
argument checks), which otherwise dominates the short layer GEMMs at M = 16.

Inputs (activations X, hidden states H, draft block) live in one device
buffer mirrored by one pinned host buffer, and the results (accept_len,
bonus, argmax) in one device buffer mirrored by one pinned host buffer, so
the host path is one graph: a copy kernel that reads the pinned inputs (a
kernel, not a copy-engine transfer, so that the step's first GEMM starts
requesting its weights while the inputs arrive) and the step, whose accept
kernel writes the results straight into the pinned host buffer (the device
addresses page-locked memory in place).

PagedVerifyStep is one layer's step over a paged 4-bit key/value cache: pages for
the draft tree, the layer's products and attention, acceptance, log probabilities
of what is answered, commit of the accepted path and the pages given back.
"""
from __future__ import annotations

import torch

from . import w12


class VerifyStep:
    def __init__(self, layers: list[w12.W12Weights], head: w12.W12Weights, B: int = 1, T: int = 16,
                 T_rows: int | None = None, device=None, grouped: bool = True):
        self.dev = torch.device(device or "cuda")
        self.B, self.T = B, T
        self.T_rows = T if T_rows is None else T_rows
        self.M = B * self.T_rows
        self.layers = layers
        self.head = head
        M = self.M
        # Input layout (byte offsets, 256-aligned): X[0..L), H, draft.
        shapes = [((M, w.K), torch.bfloat16) for w in layers] + [((M, head.K), torch.bfloat16), ((B, T), torch.int32)]
        offs, off = [], 0
        for shp, dt in shapes:
            offs.append(off)
            off += -(-shp[0] * shp[1] * (2 if dt == torch.bfloat16 else 4) // 256) * 256
        self._in_dev = torch.zeros(off, dtype=torch.uint8, device=self.dev)
        self._in_host = torch.zeros(off, dtype=torch.uint8).pin_memory()

        def carve(buf):
            return [buf[o:o + shp[0] * shp[1] * (2 if dt == torch.bfloat16 else 4)].view(dt).view(shp)
                    for o, (shp, dt) in zip(offs, shapes)]

        *self.X, self.H, self.draft = carve(self._in_dev)
        *self._X_host, self._H_host, self._draft_host = carve(self._in_host)
        self.Y = [torch.empty((M, w.N), dtype=torch.float32, device=self.dev) for w in layers]
        self.ws = [w12.workspace(w12.gemm_ws_bytes(M, w.N, w.K), self.dev) for w in layers]
        self.hws = w12.workspace(w12.verify_ws_bytes(M, head.N), self.dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.dev)
        # Results: [accept_len (B) | bonus (B) | argmax (M)] int32.
        self._out_dev = torch.zeros(2 * B + M, dtype=torch.int32, device=self.dev)
        self._out_host = torch.zeros(2 * B + M, dtype=torch.int32).pin_memory()
        self.accept_len, self.bonus, self.argmax = self._out_dev[:B], self._out_dev[B:2 * B], self._out_dev[2 * B:]
        self._results_host = (self._out_host[:B], self._out_host[B:2 * B], self._out_host[2 * B:])
        # All layer GEMMs in one launch (up to 4 per launch).
        self.groups = ([w12.Grouped([(x, w, y) for x, w, y in zip(self.X[i:i + 4], layers[i:i + 4], self.Y[i:i + 4])],
                                    M, status=self.status) for i in range(0, len(layers), 4)]
                       if grouped and layers else None)
        self.graph = None
        self.graph_host = None

    @property
    def packed_bytes(self) -> int:
        """Weight bytes (planes + group offsets) streamed by one step."""
        return sum(w.nbytes for w in self.layers) + self.head.nbytes

    @property
    def launches(self) -> int:
        """Kernel launches per step: the layer GEMMs, the fused head GEMM and its reduce/accept kernel."""
        return (len(self.groups) if self.groups is not None else len(self.layers)) + 2

    def run(self, out=None):
        """Enqueue one step on the current stream (eager libw12 calls). out:
        (accept_len, bonus, argmax) to write instead of the device results."""
        if self.groups is not None:
            for g in self.groups:
                g.run()
        else:
            for x, w, y, ws in zip(self.X, self.layers, self.Y, self.ws):
                w12.gemm(x, w, Y=y, ws=ws, status=self.status)
        w12.verify_greedy_fused(self.H, self.head, self.draft, self.T_rows, ws=self.hws, status=self.status,
                                out=out if out is not None else (self.accept_len, self.bonus, self.argmax))

    def capture(self):
        """Record one step into a CUDA graph (after one eager warm-up call)."""
        self.run()
        torch.cuda.synchronize(self.dev)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run()
        torch.cuda.synchronize(self.dev)
        self.graph = g
        return self

    def replay(self):
        if self.graph is None:
            self.capture()
        self.graph.replay()

    def host_inputs(self):
        """Pinned host views (X list, H, draft) that run_host copies in.

        Writing the next step's inputs here saves run_host a host-side copy.
        """
        return self._X_host, self._H_host, self._draft_host

    def capture_host(self):
        """Record copy-in and the step into one CUDA graph; the accept kernel
        writes its results straight into the pinned host buffer."""
        w12.copy(self._in_dev, self._in_host)
        self.run(out=self._results_host)
        torch.cuda.synchronize(self.dev)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            w12.copy(self._in_dev, self._in_host)
            self.run(out=self._results_host)
        torch.cuda.synchronize(self.dev)
        self.graph_host = g
        return self

    def run_host(self, xs_host=None, H_host=None, draft_host=None):
        """One end-to-end step from pinned host inputs to host results.

        Inputs given here are first copied into the pinned staging buffer
        (host_inputs(); pass None for any already written there). One graph
        then copies the staging buffer to the device, runs the step and copies
        (accept_len, bonus, argmax) back. Returns host tensors, valid after
        the current stream synchronises; the next run_host overwrites them.
        """
        if xs_host is not None:
            for dst, src in zip(self._X_host, xs_host):
                if src.data_ptr() != dst.data_ptr():
                    dst.copy_(src)
        for dst, src in ((self._H_host, H_host), (self._draft_host, draft_host)):
            if src is not None and src.data_ptr() != dst.data_ptr():
                dst.copy_(src)
        if self.graph_host is None:
            self.capture_host()
        self.graph_host.replay()
        return self._results_host

    def h2d_bytes(self) -> int:
        return self._in_host.numel()

    def d2h_bytes(self) -> int:
        return self._out_host.numel() * 4


class PagedVerifyStep:
    """A tree-verify step of one target layer over a paged 4-bit cache.

    B requests of T draft nodes (B * T <= 256 rows). qkv, out and head are packed
    weights: hidden -> (Hq + 2 Hkv) * head_dim, Hq * head_dim -> hidden, hidden ->
    vocabulary. Position encodings, norms and the MLP are the caller's: the step
    takes the rows that enter the layer. length int32 [B] holds each request's
    committed tokens and is advanced by every step.

    A request that there are no pages for, or whose tokens would pass max_len, is
    not served by a step: its length, pages and cached rows stay as they are, and
    the status word (int32 [1], set once, cleared by the caller) says
    W12_ERR_WORKSPACE or W12_ERR_ARG. The other requests are served as ever.
    """

    def __init__(self, qkv: w12.W12Weights, out: w12.W12Weights, head: w12.W12Weights, B: int, T: int, Hq: int,
                 Hkv: int, head_dim: int, n_pages: int, page_size: int = 64, max_len: int = 8192, top_k: int = 8,
                 device=None):
        dev = torch.device(device or "cuda")
        if qkv.N != (Hq + 2 * Hkv) * head_dim or out.K != Hq * head_dim or head.K != out.N:
            raise ValueError("qkv, out and head do not fit the heads")
        self.B, self.T, self.M, self.Hq, self.Hkv, self.head_dim = B, T, B * T, Hq, Hkv, head_dim
        self.max_len = max_len
        self.qkv, self.out, self.head, self.top_k = qkv, out, head, top_k
        self.cache = w12.KV4Cache.create(n_pages, Hkv, head_dim, page_size, dev)
        self.pages = w12.PageTable.create(B, -(-max_len // page_size), n_pages, page_size, dev)
        self.length = torch.zeros(B, dtype=torch.int32, device=dev)
        self.nodes = torch.full((B,), T, dtype=torch.int32, device=dev)
        self.attention = w12.KV4Attention(B, T, Hq, Hkv, head_dim, page_size, max_len, dev)
        self.logprobs = w12.TokenLogprobs(self.M, head.N, top_k, dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._ws = [w12.workspace(w12.gemm_ws_bytes(self.M, w.N, w.K), dev) for w in (qkv, out, head)]
        self._vws = w12.workspace(w12.verify_ws_bytes(self.M, head.N), dev)

    def prefill(self, K: torch.Tensor, V: torch.Tensor, length: torch.Tensor):
        """Cache the first length[b] rows of K, V [B, n, Hkv, head_dim] (one prompt a request).

        length int32 [B]: a request with -1 stays as it is, 0 ends one and frees its
        pages. A prompt that there are no pages for, or that is longer than n or
        max_len, leaves its request as it was and sets the status word.
        """
        n = K.shape[1]
        keep = length < 0
        # (A kept request asks for no more than it has; a count of -1 is refused.)
        start = torch.where(keep, self.length, 0)
        new = torch.where(keep, 0, torch.where(length <= self.max_len, length, -1))
        slots = self.pages.reserve(start, new, n, status=self.status)
        self.cache.append(K.flatten(0, 1), V.flatten(0, 1), slots, status=self.status)
        given = (new == 0) | (slots[:, :1] >= 0).any(1)
        self.length.copy_(torch.where(given & ~keep, length, self.length))

    def run(self, X: torch.Tensor, parents: torch.Tensor, draft: torch.Tensor) -> dict:
        """One step on X bf16 [B * T, hidden], the draft trees parents, draft int32 [B, T].

        Returns path [B, T], path_len, accept_len, bonus (as verify_tree); tokens
        [B, T], the answered tokens in order (the accepted drafts, then the bonus
        token, -1 after it), and at the same places logprob, entropy, top_logprob
        and top_id of the rows that predicted them. A request that is not served
        has path, bonus and tokens of -1 and path_len and accept_len 0.
        """
        B, T, M, d = self.B, self.T, self.M, self.head_dim
        st = self.status
        # (A negative count is refused: the request keeps its pages and gets slots of -1.)
        nodes = torch.where(self.length <= self.max_len - T, self.nodes, -1)
        slots = self.pages.reserve(self.length, nodes, T, status=st)
        served = slots[:, 0] >= 0
        Y = w12.gemm(X, self.qkv, ws=self._ws[0], status=st)
        q, k, v = Y.split([self.Hq * d, self.Hkv * d, self.Hkv * d], 1)
        # Keys and values are quantised straight from the fp32 product (views of it).
        self.cache.append(k.unflatten(1, (self.Hkv, d)), v.unflatten(1, (self.Hkv, d)), slots, status=st)
        O = self.attention.run(q.to(torch.bfloat16).view(B, T, self.Hq, d), self.cache, self.pages.table, self.length,
                               parents=parents, q_len=torch.where(served, nodes, 0), status=st)
        H = w12.gemm(O.view(M, self.Hq * d), self.out, ws=self._ws[1], status=st).to(torch.bfloat16)
        logits = w12.gemm(H, self.head, ws=self._ws[2], status=st)
        path, path_len, accept_len, bonus, _ = w12.verify_tree(logits, parents, draft, ws=self._vws, status=st)
        path, bonus = torch.where(served[:, None], path, -1), torch.where(served, bonus, -1)
        path_len, accept_len = path_len * served, accept_len * served
        # Row path[i] predicted the draft of path[i + 1], the last row of the path the bonus token.
        step = torch.arange(T, device=X.device)[None]
        nxt = torch.cat([path[:, 1:], path[:, :1]], 1).clamp(min=0).long()
        tokens = torch.where(step < accept_len[:, None], draft.gather(1, nxt), bonus[:, None])
        tokens = torch.where(step <= accept_len[:, None], tokens, -1).to(torch.int32)
        # The token asked of each row: the answered one on the path, none (-1) elsewhere.
        asked = torch.full((B, T + 1), -1, dtype=torch.int32, device=X.device)
        asked.scatter_(1, torch.where(path >= 0, path, T).long(), tokens)
        asked = asked[:, :T].contiguous()
        rows = path.clamp(min=0).long()
        lp, entropy, _, top_lp, top_id = self.logprobs.run(logits, asked.view(M, 1), status=st)
        new_len = w12.kv4_commit([self.cache], self.pages.table, self.length, path, path_len, status=st)
        self.pages.trim(new_len, status=st)
        self.length.copy_(new_len)

        def answered(t):  # rows of the path, in its order
            t = t.view(B, T, -1)
            return t.gather(1, rows[:, :, None].expand(B, T, t.shape[2]))
        return dict(path=path, path_len=path_len, accept_len=accept_len, bonus=bonus, tokens=tokens,
                    logprob=answered(lp)[..., 0], entropy=answered(entropy)[..., 0], top_logprob=answered(top_lp),
                    top_id=answered(top_id))
