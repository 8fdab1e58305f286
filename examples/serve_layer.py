"""Serves one GPT decoder layer from a paged key/value cache.

The layer that ``tp3d_layer_fwd`` trains computes whole sequences.  Here the
same parameters, in the same cube layouts, answer token by token: every step
plans the pages of its new tokens (``tp3d_paged_plan``), runs the QKV product
on the cube (``tp3d_linear``), writes keys and values into the cache
(``tp3d_paged_store``), attends over it (``tp3d_paged_attn``) and runs the
output projection and the MLP block.  Layer normalisation and the residual
sums are plain torch here.

    python examples/serve_layer.py

feeds two sequences through the server in prompt chunks and single tokens and
compares the answers with one ``tp3d_layer_fwd`` over the whole sequences.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tensor_transformer_layer_cube_gb300 as tp  # noqa: E402


class LayerServer:
    """One decoder layer on a q-cube behind a paged cache.

    ``params``: the layer's parameters in the layouts of ``tp3d_layer_fwd``
    (CUDA tensors); ``pages`` pages of ``page`` tokens serve up to ``requests``
    requests of up to ``max_tokens`` tokens.
    """

    def __init__(self, ctx, q, hidden, heads, ffn, params, requests, max_tokens, pages, page=16, eps=1e-5):
        self.ctx, self.q, self.h, self.heads, self.f, self.eps = ctx, q, hidden, heads, ffn, eps
        self.d, self.page, self.w, self.requests = hidden // heads, page, params, requests
        dev, i32 = "cuda", torch.int32
        self.k, self.v = (torch.zeros(pages, page, heads, self.d, dtype=torch.bfloat16, device=dev) for _ in range(2))
        self.cache = tp.kv_cache(self.k, self.v)
        self.free = torch.arange(pages, dtype=i32, device=dev)
        self.table = torch.full((requests, -(-max_tokens // page)), -1, dtype=i32, device=dev)
        # two of each count: a step reads one and writes the other
        self.kv_len = [torch.zeros(requests, dtype=i32, device=dev) for _ in range(2)]
        self.free_count = [torch.full((1,), pages, dtype=i32, device=dev) for _ in range(2)]
        self.q_start = torch.zeros(requests + 1, dtype=i32, device=dev)
        self.now = 0
        n = tp.tp3d_paged_attn_workspace_bytes(ctx, self.cache, heads)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=dev)

    def _norm(self, x, gamma, beta):
        y = torch.nn.functional.layer_norm(x.float(), (self.h,), self.w[gamma].float(), self.w[beta].float(), self.eps)
        return y.bfloat16()

    def _reshard(self, x, rows, cols, src, dst):
        out = torch.empty_like(x)
        tp.check(tp.tp3d_reshard(self.ctx, rows, cols, 2, src, x, dst, out), "tp3d_reshard")
        return out

    def _linear(self, x, rows, n, k, y, weight, bias):
        """x (rows x n, dense) through the cube linear with input group y; a dense rows x k."""
        cube_in, cube_out = (tp.CUBE_A, tp.CUBE_C) if y == 0 else (tp.CUBE_C, tp.CUBE_A)
        dense = tp.layout(tp.ROW, 0, 1)
        out = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda")
        xin = self._reshard(x, rows, n, dense, tp.layout(cube_in, self.q))
        tp.check(tp.tp3d_linear(self.ctx, self.q, y, rows, n, k, tp.TP3D_BF16, xin, self.w[weight], self.w[bias], 0,
                                out), "tp3d_linear")
        return self._reshard(out, rows, k, tp.layout(cube_out, self.q), dense)

    def step(self, x, fresh):
        """The layer's output for the new tokens: ``x`` (sum(fresh) x hidden,
        request by request), ``fresh`` the number of each request's."""
        tokens, h, d = x.shape[0], self.h, self.d
        unit = 8 * self.q * self.q  # the cube's shards have a multiple of 8 rows: pad
        rows = -(-tokens // unit) * unit
        x = torch.cat([x, x.new_zeros(rows - tokens, h)])
        slots = torch.empty(rows, dtype=torch.int64, device="cuda")
        positions = torch.empty(rows, dtype=torch.int32, device="cuda")
        a, b = self.now, 1 - self.now
        tp.check(tp.tp3d_paged_plan(self.ctx, self.page, self.requests, rows, self.kv_len[a],
                                    torch.tensor(fresh, dtype=torch.int32, device="cuda"), self.free,
                                    self.free.numel(), self.free_count[a], self.table, self.table.shape[1],
                                    self.q_start, self.kv_len[b], slots, positions, self.free_count[b]),
                 "tp3d_paged_plan")
        qkv = self._linear(self._norm(x, "ln1_g", "ln1_b"), rows, h, 3 * h, 0, "w_qkv", "b_qkv")
        q, k, v = (qkv[:, i * h:(i + 1) * h].view(rows, self.heads, d) for i in range(3))
        tp.check(tp.tp3d_paged_store(self.ctx, self.cache, k, v, slots), "tp3d_paged_store")
        batch = tp.paged_batch(self.q_start, self.kv_len[b], self.table, rows, max(fresh))
        o = torch.zeros(rows, self.heads, d, dtype=torch.bfloat16, device="cuda")
        tp.check(tp.tp3d_paged_attn(self.ctx, self.cache, batch, q, o, None, d ** -0.5, self.workspace),
                 "tp3d_paged_attn")
        y = (x.float() + self._linear(o.view(rows, h), rows, h, h, 1, "w_o", "b_o").float()).bfloat16()
        cube_a, dense = tp.layout(tp.CUBE_A, self.q), tp.layout(tp.ROW, 0, 1)
        z = self._reshard(self._norm(y, "ln2_g", "ln2_b"), rows, h, dense, cube_a)
        y1 = torch.empty(rows * self.f, dtype=torch.bfloat16, device="cuda")
        out = torch.empty_like(z)
        tp.check(tp.tp3d_mlp(self.ctx, self.q, rows, h, self.f, tp.TP3D_BF16, z, self.w["w_1"], self.w["b_1"],
                             self.w["w_2"], self.w["b_2"], y1, out), "tp3d_mlp")
        out = self._reshard(out, rows, h, cube_a, dense)
        self.now = b
        return (y.float() + out.float()).bfloat16()[:tokens]


def compare(q=2, batch=2, seq=256, hidden=256, heads=2, ffn=1024, chunks=((100, 61), (1, 1), (90, 130), (64, 63)),
            seed=7):
    """Feeds ``batch`` sequences to a server, ``chunks`` first and the rest one
    token at a time.  Returns the answers and tp3d_layer_fwd's, dense
    (batch * seq x hidden)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(n, std, mean=0.0):
        return (torch.randn(n, generator=gen, device="cuda") * std + mean).bfloat16()

    # random parameters: their layout on the cube is only an order of theirs
    h, f = hidden, ffn
    sizes = {"w_qkv": 3 * h * h, "w_o": h * h, "w_1": h * f, "w_2": f * h, "b_qkv": 3 * h, "b_o": h, "b_1": f, "b_2": h,
             "ln1_b": h, "ln2_b": h}
    params = {k: normal(n, 0.02 if k[0] != "w" else 0.05) for k, n in sizes.items()}
    params |= {k: normal(h, 0.02, 1.0) for k in ("ln1_g", "ln2_g")}
    ctx = tp.tp3d_create(torch.cuda.current_device())
    try:
        x = normal(batch * seq * h, 1.0).view(batch * seq, h)
        server = LayerServer(ctx, q, h, heads, f, params, batch, seq, batch * (seq // 16) + 1)
        cfg = tp.tp3d_layer_cfg(q, batch, seq, h, heads, f, tp.TP3D_BF16, server.eps)
        ws = torch.empty(tp.tp3d_layer_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
        cube_a, dense = tp.layout(tp.CUBE_A, q), tp.layout(tp.ROW, 0, 1)
        whole = torch.empty_like(x)
        tp.check(tp.tp3d_layer_fwd(ctx, cfg, params, server._reshard(x, batch * seq, h, dense, cube_a), whole, ws))
        whole = server._reshard(whole, batch * seq, h, cube_a, dense)

        x3, have = x.view(batch, seq, h), [0] * batch
        answers = torch.empty_like(x3)
        steps = list(chunks)
        while min(have) < seq:
            fresh = list(steps.pop(0)) if steps else [int(n < seq) for n in have]
            y = server.step(torch.cat([x3[b, n:n + k] for b, (n, k) in enumerate(zip(have, fresh))]), fresh)
            at = 0
            for b, k in enumerate(fresh):
                answers[b, have[b]:have[b] + k] = y[at:at + k]
                at, have[b] = at + k, have[b] + k
        tp.check(tp.tp3d_sync_status(ctx), "device")
        return answers.view(batch * seq, h), whole
    finally:
        tp.tp3d_destroy(ctx)


if __name__ == "__main__":
    got, want = (t.float() for t in compare())
    print("largest difference %.3g of the largest answer %.3g" % (float((got - want).abs().max()), float(want.abs().max())))
