"""Users encoded from their histories: item rows from an embedding table, layer norm, one projection to queries, keys
and values, attention of each history over itself with a learned bias by relative position, a projection back, dropout
and the rows added again. Histories come without padding; for serving their keys and values are kept in a paged cache,
and a user's new item is encoded alone.

    python -m dlrm_sparse_embedding_amd.history [--users N --history N --steps N]

takes training steps on synthetic histories, serves new items of the same users and prints what each took.
"""
from __future__ import annotations

import argparse
import math

import torch

from . import emb as E
from .ranking import Pages


class HistoryEncoder(Pages):
    """One layer over embedded items. A distance of `exact` items and more shares its bias with others, from near `far`
    on with all (emb.HistoryAttention); with no buckets there is no bias. Its weights are fp32, those of the two projections with a rounded copy."""

    def __init__(self, items: int, width: int = 128, heads: int = 8, kv_heads: int = 2, dim: int = 64,
                 buckets: int = 32, exact: int = 16, far: int = 1024, dropout: float = 0.1, pages: int = 1024,
                 page: int = 16, seed: int = 0, dtype=torch.bfloat16):
        self.heads, self.kv_heads, self.dim, self.eps, self.dtype = heads, kv_heads, dim, 1e-5, dtype
        self.dropout, self.seed = dropout, seed
        self.tables = E.EmbeddingTables([E.TableSpec(items, width, "f32")], with_state=True)
        self.tables.init_uniform(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.norm_w, self.norm_b = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
        out = (heads + 2 * kv_heads) * dim
        self.master = torch.randn((width, out), generator=gen, device="cuda").mul_(1 / math.sqrt(width))
        self.back_master = torch.randn((heads * dim, width), generator=gen, device="cuda").mul_(1 / math.sqrt(heads * dim))
        self.proj, self.back = self.master.to(dtype), self.back_master.to(dtype)
        self.attention = E.HistoryAttention(heads, kv_heads, dim, "bf16" if dtype == torch.bfloat16 else "f16",
                                            buckets=buckets, exact=exact if buckets else 0, far=far if buckets else 0)
        self.bias = torch.zeros((self.attention.bias_rows, heads), device="cuda") if buckets else None
        self.count = torch.zeros(1, dtype=torch.int64, device="cuda")     # training steps taken: dropout's step
        self.hold_cache(pages, page, kv_heads, dim, dtype)

    def close(self) -> None:
        self.tables.close()
        self.attention.close()
        self.cache.close()

    def rows(self, ids: torch.Tensor) -> torch.Tensor:
        """The items' rows [n, width], fp32."""
        return self.tables.forward(ids, self._bags(ids), ids.numel(), "sum")

    def _bags(self, ids):
        return torch.arange(ids.numel() + 1, dtype=ids.dtype, device=ids.device)

    def parts(self, fused):
        h, k = self.heads, self.kv_heads
        return fused[:, :h], fused[:, h:h + k], fused[:, h + k:]

    def _fused(self, rows):
        """The rows normed, and their queries, keys and values [n, heads + 2 kv_heads, dim]."""
        normed = torch.empty_like(rows, dtype=self.dtype)
        E.emb_layer_norm(rows, normed, self.norm_w, self.norm_b, self.eps)
        return normed, (normed @ self.proj).view(rows.shape[0], self.heads + 2 * self.kv_heads, self.dim)

    def _workspace(self, need):
        # a call's own: calls on other streams may be under way
        return torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

    # ---- training ----

    def forward(self, rows, offsets, train: bool = False):
        """The histories' rows [n, width], those of user u offsets[u] .. offsets[u + 1] (int32), encoded: [n, width] of
        the layer's type, and what `backward` needs. train: with dropout, whose mask `count` chooses."""
        normed, fused = self._fused(rows)
        out = torch.empty((rows.shape[0], self.heads, self.dim), dtype=self.dtype, device="cuda")
        lse = torch.empty(out.shape[:2], device="cuda")
        E.emb_history_attention(self.attention.handle, *self.parts(fused), out, offsets, bias=self.bias, lse=lse)
        y = out.flatten(1) @ self.back
        # the rows join in the layer's type, as dropout takes operands of one type: half a step of them, next to that of
        # the sum, which is stored in it anyway
        E.emb_dropout(y, y, self.dropout if train else 0.0, self.seed, step=self.count, residual=rows.to(self.dtype))
        return y, (rows, offsets, normed, fused, out, lse)

    def backward(self, saved, dy):
        """Gradients, from that of the encoded rows dy [n, width] of the layer's type, of the rows and the weights: a
        dict with "rows", "proj", "back", "norm_w", "norm_b", "bias". `count` is still the forward's; the forward was
        one with train."""
        rows, offsets, normed, fused, out, lse = saved
        d_back = torch.empty_like(dy)
        E.emb_dropout(dy, d_back, self.dropout, self.seed, step=self.count)
        d_out = (d_back @ self.back.t()).view_as(out)
        g = torch.empty_like(fused)
        d_bias = None if self.bias is None else torch.empty_like(self.bias)
        ws = self._workspace(E.emb_history_attention_workspace_bytes(self.attention.handle, rows.shape[0],
                                                                     offsets.numel() - 1))
        E.emb_history_attention_backward(self.attention.handle, *self.parts(fused), out, lse, d_out, *self.parts(g),
                                         offsets, ws, bias=self.bias, dbias=d_bias)
        g = g.flatten(1)
        d_normed = g @ self.proj.t()
        d_rows = torch.empty_like(rows)
        d_w, d_b = torch.empty_like(self.norm_w), torch.empty_like(self.norm_b)
        ws = self._workspace(E.emb_layer_norm_workspace_bytes(*rows.shape))
        E.emb_layer_norm_backward(rows, d_normed, d_rows, self.norm_w, self.eps, ws, d_w, d_b)
        return {"rows": d_rows.add_(dy), "proj": normed.t() @ g, "back": out.flatten(1).t() @ d_back, "norm_w": d_w,
                "norm_b": d_b, "bias": d_bias}

    def train_step(self, ids, offsets, gradient, lr: float) -> torch.Tensor:
        """One step of the items' rows and the layer's weights on the histories' items; `gradient` maps the encoded
        rows to their gradient. Returns the encoded rows."""
        y, saved = self.forward(self.rows(ids), offsets, train=True)
        d = self.backward(saved, gradient(y))
        self.count += 1
        for master, copy, name in ((self.master, self.proj, "proj"), (self.back_master, self.back, "back")):
            master -= lr * d[name].float()
            copy.copy_(master)
        for weight, name in ((self.norm_w, "norm_w"), (self.norm_b, "norm_b"), (self.bias, "bias")):
            if weight is not None:
                weight -= lr * d[name]
        bufs = self.tables.backward_buffers(ids.numel(), ids.numel(), with_grad=False)
        self.tables.backward(ids, self._bags(ids), ids.numel(), "sum", d["rows"], bufs)
        self.tables.update("adagrad", lr, 1e-8, bufs, dY=d["rows"])
        return y

    # ---- serving ----

    def append(self, ids, offsets, lens, table):
        """Encodes whole histories and writes their keys and values to their pages (lens, table: emb_kv_append)."""
        y, (_, _, _, fused, _, _) = self.forward(self.rows(ids), offsets)
        _, k, v = self.parts(fused)
        E.emb_kv_append(self.cache.handle, None, k, v, offsets, lens, table)
        return y

    def step(self, ids, lens, table):
        """Encodes one new item of each user: [users, width]. lens (int32) counts it, table has a page for it, and the
        user's earlier items were appended."""
        rows = self.rows(ids)
        _, fused = self._fused(rows)
        q, k, v = self.parts(fused)
        E.emb_kv_append(self.cache.handle, None, k, v, None, lens, table)
        out = torch.empty((rows.shape[0], self.heads, self.dim), dtype=self.dtype, device="cuda")
        ws = self._workspace(E.emb_history_step_workspace_bytes(self.attention.handle, self.cache.handle, rows.shape[0],
                                                                table.shape[1]))
        E.emb_history_step(self.attention.handle, self.cache.handle, q, out, lens, table, ws, bias=self.bias)
        y = out.flatten(1) @ self.back
        E.emb_dropout(y, y, 0.0, self.seed, residual=rows.to(self.dtype))
        return y


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--users", type=int, default=64)
    ap.add_argument("--history", type=int, default=600, help="the longest history")
    ap.add_argument("--steps", type=int, default=3)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(1)
    items = 100000
    r = HistoryEncoder(items, pages=a.users * (-(-(a.history + a.steps) // 16)))

    def timed(what, f):
        start, end = torch.cuda.Event(True), torch.cuda.Event(True)
        start.record()
        out = f()
        end.record()
        end.synchronize()
        print(f"{what}: {start.elapsed_time(end):.3f} ms")
        return out

    counts = torch.randint(1, a.history + 1, (a.users,), generator=gen, device="cuda")
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    n = int(offsets[-1])
    ids = torch.randint(0, items, (n,), generator=gen, device="cuda")
    target = torch.randn((n, 128), generator=gen, device="cuda")
    for _ in range(a.steps):      # the first calls load kernels
        timed(f"training step on {n} items of {a.users} users",
              lambda: r.train_step(ids, offsets, lambda y: (2 / n * (y.float() - target)).to(y.dtype), lr=0.01))
    lens = counts.to(torch.int32)
    table = r.new_pages((counts + a.steps).tolist())
    timed(f"append {n} items", lambda: r.append(ids, offsets, lens, table))
    for _ in range(a.steps):
        lens = lens + 1
        new = torch.randint(0, items, (a.users,), generator=gen, device="cuda")
        out = timed(f"one new item of {a.users} users", lambda: r.step(new, lens, table))
    r.cache.check_error()
    r.attention.check_error()
    r.tables.check_device_error()
    print(f"mean |output| {out.float().abs().mean().item():.4f}")
    r.close()


if __name__ == "__main__":
    main()
