"""The layer operators on the GPU at the places where they once went wrong, and on paths of their own."""
from __future__ import annotations

import pytest
import torch

import layer_ref as ref
import mixed_precision_partial_amd as ar
import test_layer_gpu as base
from gpu_util import log_case

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    c = ar.ar_init(0)
    yield c
    torch.cuda.synchronize()
    ar.ar_free(c)


@pytest.mark.parametrize("keys", [1, 700])
def test_attention_of_one_row_of_head_major_buffers(ctx, keys):
    """Queries, output, keys and values of one token between 70000 others of the same head."""
    log_case(f"head-major rows, {keys} keys")
    q, k, v, _, _, kl = base.attn_case(BF16, [1], [keys], 16, 2, 128)
    q, cu = q[:1], torch.tensor([0, 1], dtype=torch.int32)
    wide_q = torch.zeros(2, 16, 70000, 128, dtype=BF16, device="cuda")
    wide_k = torch.full((2, 2, 70000, 128), float("nan"), dtype=BF16, device="cuda")
    dq, out = wide_q[0][:, 6:7].transpose(0, 1), wide_q[1][:, 60000:60001].transpose(0, 1)
    dk, dv = (wide_k[i][:, 9:9 + keys].transpose(0, 1) for i in (0, 1))
    dq.copy_(q)
    dk.copy_(k)
    dv.copy_(v)
    lse = torch.empty(1, 16, device="cuda")
    ar.ar_attention(ctx, out, dq, dk, dv, cu.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda"), kl.cuda(), 1, keys, lse=lse)
    torch.cuda.synchronize()
    want, wl, tol, tl = ref.attention(q, k, v, cu, [0], kl, True, 128 ** -0.5)
    base.near(out, want, tol, "one row")
    base.near(lse, wl, tl, "one row's lse")
    out.zero_()
    assert not bool(wide_q[1].any())
