"""Candidates ranked against users' histories: item rows from an embedding
table, queries, keys and values from one projection of them, the histories'
keys and values in a paged cache that is written once, and every candidate
attending to its user's whole history and to itself.

    python -m dlrm_sparse_embedding_amd.ranking [--users N --history N --candidates N]

appends synthetic histories, ranks candidates, takes a training step on the
projection's inputs and prints what each took.
"""
from __future__ import annotations

import argparse
import math

import torch

from . import emb as E


class Pages:
    """A paged cache and who has its pages."""

    def hold_cache(self, pages: int, page: int, kv_heads: int, dim: int, dtype) -> None:
        shape = (pages, kv_heads, page, dim)       # a page holds each head's rows together
        self.page = page
        self.cache = E.KVCache(torch.zeros(shape, dtype=dtype, device="cuda").transpose(1, 2),
                               torch.zeros(shape, dtype=dtype, device="cuda").transpose(1, 2))
        self.next_page = 0        # pages from here on were never handed out
        self.returned = []        # pages handed back

    def new_pages(self, counts) -> torch.Tensor:
        """A page table row for each of `counts` slots; -1 behind the last page."""
        need = [-(-int(c) // self.page) for c in counts]
        if sum(need) > len(self.returned) + self.cache.pages - self.next_page:
            raise ValueError("the cache has no pages left")
        table = torch.full((len(need), max(need + [1])), -1, dtype=torch.int32)
        for row, n in zip(table, need):
            again = min(n, len(self.returned))
            if again:
                row[:again] = torch.tensor(self.returned[-again:], dtype=torch.int32)
                del self.returned[-again:]
            row[again:n] = torch.arange(self.next_page, self.next_page + n - again, dtype=torch.int32)
            self.next_page += n - again
        return table.cuda()

    def return_pages(self, table) -> None:
        """Hands back the pages of new_pages' table rows, for later rows. Work on them has to be done, or under way
        on the stream that will use them next."""
        pages = [p for p in table.flatten().tolist() if p >= 0]
        if len(set(pages)) != len(pages) or any(p >= self.next_page for p in pages) or set(pages) & set(self.returned):
            raise ValueError("a page that is not handed out")
        self.returned += pages


class HistoryRanker(Pages):
    """One attention layer over embedded items. Positions are places in a history; a candidate takes the place
    after its last item. With ``norm`` queries and keys are normed per head, otherwise only turned."""

    def __init__(self, items: int, width: int = 64, heads: int = 8, kv_heads: int = 2, dim: int = 64,
                 pages: int = 1024, page: int = 16, norm: bool = True, layout: str = "half", seed: int = 0,
                 dtype=torch.bfloat16):
        self.heads, self.kv_heads, self.dim, self.eps = heads, kv_heads, dim, 1e-6
        self.dtype = dtype
        self.tables = E.EmbeddingTables([E.TableSpec(items, width, "f32")], with_state=True)
        self.tables.init_uniform(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        out = (heads + 2 * kv_heads) * dim
        # Steps are taken on fp32 weights, most of them being less than half a step of a 16-bit one; proj is their
        # rounded copy, written after each. Weights from elsewhere go into both.
        self.master = torch.randn((width, out), generator=gen, device="cuda").mul_(4 / math.sqrt(width))
        self.proj = self.master.to(dtype)
        self.wq = torch.ones(dim, device="cuda") if norm else None
        self.wk = torch.ones(dim, device="cuda") if norm else None
        self.norm = norm
        self.rotary = E.Rotary(dim, layout=layout)
        self.hold_cache(pages, page, kv_heads, dim, dtype)

    def close(self) -> None:
        self.tables.close()
        self.rotary.close()
        self.cache.close()

    # ---- items to queries, keys and values ----

    def rows(self, ids: torch.Tensor) -> torch.Tensor:
        """The items' rows [n, width], fp32."""
        return self.tables.forward(ids, self._bags(ids), ids.numel(), "sum")

    def _bags(self, ids):
        return torch.arange(ids.numel() + 1, dtype=ids.dtype, device=ids.device)

    def project(self, rows: torch.Tensor) -> torch.Tensor:
        """[n, heads + 2 kv_heads, dim]: queries, keys, values."""
        return (rows.to(self.dtype) @ self.proj).view(rows.shape[0], self.heads + 2 * self.kv_heads, self.dim)

    def parts(self, fused):
        h, k = self.heads, self.kv_heads
        return fused[:, :h], fused[:, h:h + k], fused[:, h + k:]

    def place(self, q, k, positions):
        """Queries (and keys, or None) normed, if the ranker does, and turned to their positions."""
        qo, ko = torch.empty_like(q), None if k is None else torch.empty_like(k)
        if self.norm:
            E.emb_qk_norm_rotary(self.rotary.handle, positions, q, qo, k, ko, self.wq, self.wk, self.eps)
        else:
            E.emb_rotary_apply(self.rotary.handle, positions, q, qo, k, ko)
        return qo, ko

    # ---- serving ----

    def append(self, ids, offsets, lens, table, positions=None) -> None:
        """Writes the items' keys and values to their sequences' pages (offsets, lens, table: emb_kv_append)."""
        _, k, v = self.parts(self.project(self.rows(ids)))
        E.emb_kv_append(self.cache.handle, self.rotary.handle, k, v, offsets, lens, table, wk=self.wk,
                        eps=self.eps if self.norm else None, positions=positions)

    def rank(self, ids, group_offsets, history_lens, history_table, table):
        """Attention output [n, heads, dim] and its log-sum of each candidate: candidates group_offsets[u] ..
        group_offsets[u + 1] belong to user u; `table` names a page for each candidate itself."""
        n = ids.numel()
        q, k, v = self.parts(self.project(self.rows(ids)))
        user = torch.repeat_interleave(torch.arange(history_lens.numel(), device=ids.device),
                                       group_offsets.diff().long(), output_size=n)
        place = history_lens.long()[user]
        one = torch.ones(n, dtype=torch.int32, device=ids.device)
        qr, _ = self.place(q, None, place)
        E.emb_kv_append(self.cache.handle, self.rotary.handle, k, v, None, one, table, wk=self.wk,
                        eps=self.eps if self.norm else None, positions=place)
        need = E.emb_prefix_attention_workspace_bytes(self.cache.handle, n, self.heads, history_lens.numel(),
                                                      history_table.shape[1], table.shape[1])
        # a call's own: calls on other streams may be under way
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(qr)
        lse = torch.empty((n, self.heads), device="cuda")
        E.emb_prefix_attention(self.cache.handle, qr, out, 1 / math.sqrt(self.dim), None, one, table, group_offsets,
                               history_lens, history_table, ws, lse=lse)
        return out, lse

    # ---- training ----

    def place_backward(self, q, k, positions, dq, dk):
        """Gradients of `place`: of its inputs, and of the norm's weights (None without a norm)."""
        gq, gk = torch.empty_like(dq), torch.empty_like(dk)
        if not self.norm:
            E.emb_rotary_apply(self.rotary.handle, positions, dq, gq, dk, gk, inverse=True)
            return gq, gk, None, None
        dwq, dwk = torch.empty_like(self.wq), torch.empty_like(self.wk)
        n = E.emb_qk_norm_rotary_workspace_bytes(q.shape[0], self.heads, self.kv_heads, self.dim)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        E.emb_qk_norm_rotary_backward(self.rotary.handle, positions, q, dq, gq, k, dk, gk, self.wq, self.wk, self.eps,
                                      ws, dwq, dwk)
        return gq, gk, dwq, dwk

    def train_step(self, ids, positions, dq, dk, dv, lr: float) -> None:
        """One step of the items' rows, the projection and the norm's weights, given the gradients of the placed
        queries and keys and of the values."""
        rows = self.rows(ids)
        q, k, _ = self.parts(self.project(rows))
        gq, gk, dwq, dwk = self.place_backward(q, k, positions, dq, dk)
        g = torch.cat([gq, gk, dv], 1).view(ids.numel(), self.proj.shape[1])
        d_rows = (g @ self.proj.t()).float()
        # both products sum in fp32 and round once to the type of the heads
        self.master -= lr * (rows.to(self.dtype).t() @ g).float()
        self.proj.copy_(self.master)
        if self.norm:
            self.wq -= lr * dwq
            self.wk -= lr * dwk
        off = self._bags(ids)
        bufs = self.tables.backward_buffers(ids.numel(), ids.numel(), with_grad=False)
        self.tables.backward(ids, off, ids.numel(), "sum", d_rows, bufs)
        self.tables.update("adagrad", lr, 1e-8, bufs, dY=d_rows)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--users", type=int, default=8)
    ap.add_argument("--history", type=int, default=2000)
    ap.add_argument("--candidates", type=int, default=400)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(1)
    items = 100000
    pages = a.users * (-(-a.history // 16)) + a.candidates
    r = HistoryRanker(items, pages=pages)

    def timed(what, f):
        start, end = torch.cuda.Event(True), torch.cuda.Event(True)
        start.record()
        out = f()
        end.record()
        end.synchronize()
        print(f"{what}: {start.elapsed_time(end):.3f} ms")
        return out

    history = torch.randint(0, items, (a.users * a.history,), generator=gen, device="cuda")
    lens = torch.full((a.users,), a.history, dtype=torch.int32, device="cuda")
    offsets = torch.arange(0, history.numel() + 1, a.history, dtype=torch.int32, device="cuda")
    table = r.new_pages([a.history] * a.users)
    ids = torch.randint(0, items, (a.candidates,), generator=gen, device="cuda")
    groups = torch.linspace(0, a.candidates, a.users + 1, device="cuda").to(torch.int32)
    for _ in range(2):      # the first calls load kernels
        own = r.new_pages([1] * a.candidates)
        timed(f"append {history.numel()} items", lambda: r.append(history, offsets, lens, table))
        out, _ = timed(f"rank {a.candidates} candidates of {a.users} users",
                       lambda: r.rank(ids, groups, lens, table, own))
        grads = [torch.randn((ids.numel(), n, r.dim), generator=gen, device="cuda").to(r.dtype)
                 for n in (r.heads, r.kv_heads, r.kv_heads)]
        places = torch.full((ids.numel(),), a.history, dtype=torch.int64, device="cuda")
        timed("training step", lambda: r.train_step(ids, places, *grads, lr=0.01))
        r.return_pages(own)
    r.cache.check_error()
    r.tables.check_device_error()
    print(f"mean |output| {out.float().abs().mean().item():.4f}")
    r.close()


if __name__ == "__main__":
    main()
