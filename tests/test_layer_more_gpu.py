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


SMALL = [  # tokens, heads_q, heads_kv, dim, keys, the key that dominates
    (1, 8, 1, 128, 65536, 0), (1, 8, 1, 64, 65536, 40000), (2, 8, 2, 256, 20000, 19999),      # few rows
    (3, 32, 1, 128, 30000, 0), (90, 2, 1, 64, 30000, 15000), (70, 1, 1, 256, 20000, 0),       # tiles of rows
]


@pytest.mark.parametrize("case", SMALL, ids=lambda c: "-".join(map(str, c)))
def test_attention_small_probabilities_in_fp16_add_up(ctx, case):
    """One key's score is 26 powers of two above those of all others, whose values alone are not zero: the
    others' probabilities are 2^-26 of the largest each, and the result is their sum.

    An error of 2^-32 (half of binary16's smallest step, 2^-25, beside probabilities of up to 2^7 where
    the largest is the row's reference) in each of n probabilities, the binary32 sum of n of them, a few steps
    of the exponents, and the roundings of a probability and of the result."""
    tokens, hq, hkv, d, n, at = case
    log_case(f"small probabilities {case}")
    q, k = torch.zeros(tokens, hq, d, dtype=F16, device="cuda"), torch.zeros(n, hkv, d, dtype=F16, device="cuda")
    v = torch.ones(n, hkv, d, dtype=F16, device="cuda")
    q[..., 3] = 1
    k[at, :, 3] = 26 * 0.6931
    v[at] = 0
    out, lse = torch.empty_like(q), torch.empty(tokens, hq, device="cuda")
    ar.ar_attention(ctx, out, q, k, v, torch.tensor([0, tokens], dtype=torch.int32, device="cuda"),
                    torch.zeros(1, dtype=torch.int64, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda"),
                    tokens, n, causal=False, scale=1.0, lse=lse)
    torch.cuda.synchronize()
    top = k[at, :1, 3].double().cpu()
    rest = (n - 1) * torch.exp(-top)
    want, u = rest / (1 + rest), ref.U[F16]
    e = (n + 64) * ref.U32 + 8 * ref.U32 * top
    tol = 1.01 * (want * (2 * u + e) + n * 2.0 ** -32) + ref.TINY[F16]
    base.near(out, want.expand(out.shape), tol.expand(out.shape), "small probabilities")
    base.near(lse, (top + (1 + rest).log()).expand(lse.shape), (1.01 * e + 4 * ref.U32 * top).expand(lse.shape), "their lse")
