"""GPU tests of layer norm and dropout at their limits: the longest row, more rows than one launch takes, the gradient
in place of its input. Inputs are broadcast where only their number counts."""
import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E
from oracle import history_oracle as H
from tests.test_gpu_history_rows import rows_of

pytestmark = pytest.mark.gpu


def kept(row, unit, seed, threshold):
    """Of the 8 columns of a unit, in step 0."""
    words = [H.philox((unit, row, 0, second), (seed % 2 ** 32, seed >> 32)) for second in (0, 2 ** 31)]
    hi, lo = ([w[j // 2] >> 16 * (j % 2) & 0xFFFF for j in range(8)] for w in words)
    return [h << 16 | x >= threshold for h, x in zip(hi, lo)]


def test_dropout_of_the_longest_row():
    n, seed = (1 << 31) - 1, 77
    x = torch.full((1, n), 1.0, dtype=torch.bfloat16, device="cuda")
    y = torch.full_like(x, 7.0)
    E.emb_dropout(x, y, 0.5, seed)
    for unit in (0, 1 << 27, (1 << 28) - 1):
        want = [2.0 * k for k in kept(0, unit, seed, 1 << 31)]
        assert y[0, 8 * unit:8 * unit + 8].tolist() == want[:n - 8 * unit]
    assert ((y == 0) | (y == 2)).all()
    E.emb_dropout(x, y, 0.0, seed)
    assert torch.equal(x, y)


def test_dropout_of_more_rows_than_one_launch_takes():
    n, seed = (1 << 30) + 1000, 12345
    x = torch.ones((1, 1), dtype=torch.bfloat16, device="cuda").expand(n, 1)
    y = torch.full((n, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    E.emb_dropout(x, y, 0.5, seed)
    for row in [0, 1, (1 << 30) - 1, *range(1 << 30, (1 << 30) + 30), n - 1]:
        assert y[row].item() == 2.0 * kept(row, 0, seed, 1 << 31)[0]
    assert ((y == 0) | (y == 2)).all()


def test_layer_norm_of_the_most_rows():
    n = (1 << 31) - 1
    x = torch.ones((1, 1), dtype=torch.bfloat16, device="cuda").expand(n, 1)
    y = torch.full((n, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    b = torch.tensor([3.0], device="cuda")
    E.emb_layer_norm(x, y, None, b, 1e-5)
    assert (y == 3).all()


@pytest.mark.parametrize("xt,yt,rows,dim,memory", [
    ("f32", "bf16", 70, 128, "plain"), ("f32", "f16", 9001, 96, "odd"), ("f32", "f32", 9, 4096, "plain"),
    ("bf16", "bf16", 3001, 1024, "strided"), ("f16", "f16", 700, 65, "odd"), ("f32", "bf16", 300, 2047, "odd")])
def test_gradient_in_place_of_the_input(xt, yt, rows, dim, memory):
    gen = torch.Generator().manual_seed(rows + dim)
    x, dy = rows_of(gen, rows, dim, xt, memory), rows_of(gen, rows, dim, yt, memory)
    w = (1 + 0.3 * torch.randn(dim, generator=gen)).cuda()
    ws = torch.empty(E.emb_layer_norm_workspace_bytes(rows, dim), dtype=torch.uint8, device="cuda")
    want = [torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)]
    E.emb_layer_norm_backward(x, dy, want[0], w, 1e-5, ws, *want[1:])
    got = [x, torch.empty_like(w), torch.empty_like(w)]
    E.emb_layer_norm_backward(x, dy, x, w, 1e-5, ws, *got[1:])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    if memory != "plain":      # nothing beside the rows was written
        rest = x._base.clone()
        rest[:, x.storage_offset():x.storage_offset() + dim] = float("nan")
        assert rest.isnan().all()
