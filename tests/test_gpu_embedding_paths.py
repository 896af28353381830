"""The embedding and its gradient where their kernels change: more tokens than the machine has threads (several a thread),
rows wider than a block.  Tolerances as test_gpu_embedding.py derives them."""
import pytest
import torch

import param_buffers_gb300 as gtp
from test_gpu_embedding import B, DEV, F, check_gradient, check_lookup, make_ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("td,od", [(B, B), (B, F), (F, F), (F, B)])
@pytest.mark.parametrize("T,rows,C", [(2003, 300, 2048), (2003, 300, 2047), (9001, 77, 512), (70001, 50, 16), (70001, 50, 15),
                                      (1301, 40, 4104)])
def test_lookup_of_many_tokens(T, rows, C, td, od):
    ids = make_ids(T, rows, rows).to(DEV)
    table = torch.randn(rows, C + 8, device=DEV).to(td)[:, :C]
    out = torch.full((T, C), float("nan"), dtype=od, device=DEV)
    gtp.gtp_embedding(ids, table, out, first_row=rows, scale=-1.7)
    check_lookup(out, ids, table, rows, -1.7)


@pytest.mark.parametrize("dd,gd", [(B, F), (F, F), (B, B), (F, B)])
@pytest.mark.parametrize("T,rows,C", [(300, 20, 4104), (300, 20, 4099), (3001, 100, 2048), (3001, 10, 2056), (64, 5, 6152)])
def test_gradient_of_wide_rows(T, rows, C, dd, gd):
    for kind in ("mixed", "one row"):
        ids = make_ids(T, rows, 5, kind).to(DEV)
        dout, before = torch.randn(T, C, device=DEV).to(dd), torch.randn(rows * C, device=DEV).to(gd)
        grad = before.clone()
        ws = torch.empty(gtp.gtp_embedding_grad_workspace_bytes(T, rows, C), dtype=torch.uint8, device=DEV).fill_(0xFF)
        gtp.gtp_embedding_grad_accum(dout, ids, grad, 0, rows, ws, first_row=5, scale=0.3)
        check_gradient(grad, before, ids, dout, 5, rows, 0.3)
