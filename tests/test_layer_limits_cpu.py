"""The limits that ar.h states for the layer operators, from both sides, without a GPU: a call within them is
stopped by the runtime only (made-up addresses), one beyond them is refused as unsupported."""
from __future__ import annotations

import pytest

import mixed_precision_partial_amd as ar
import test_layer_cpu as base
from test_layer_cpu import fake  # noqa: F401  (a fixture)

FITS, BEYOND = ar.AR_ERR_RUNTIME, ar.AR_ERR_UNSUPPORTED
FAR = dict(q_token=1 << 12, k_token=1 << 12, v_token=1 << 12, o_token=1 << 12)


@pytest.mark.parametrize("want,change", [
    (FITS, dict(heads_q=65532, heads_kv=2, tokens=1)), (BEYOND, dict(heads_q=65533, heads_kv=2, tokens=1)),
    (FITS, dict(heads_q=4, heads_kv=2, tokens=(1 << 28) - 1, cache_rows=50)), (BEYOND, dict(heads_q=4, heads_kv=2, tokens=1 << 28)),
], ids=str)
def test_qk(fake, want, change):  # noqa: F811
    """Tensors in places of their own, far enough from each other for the largest of them."""
    t = 1 << 46
    places = {k: (1 << 44) + i * t for i, k in enumerate(("q_out", "q", "k", "v", "positions", "slots", "table", "k_out", "v_out"))}
    assert base.call_qk(fake, **{**places, **change, "q_weight": None, "k_weight": None}) == want


@pytest.mark.parametrize("want,change", [
    (FITS, dict(batch=65535, max_q=1)), (BEYOND, dict(batch=65536, max_q=1)),
    (FITS, dict(max_k=(1 << 31) - 1, rows_k=(1 << 31) - 128)), (BEYOND, dict(max_k=(1 << 31) - 1, rows_k=(1 << 31) - 127)),
    (FITS, dict(max_k=(1 << 31) - 128, rows_k=1 << 33)), (BEYOND, dict(rows_k=1 << 48)), (BEYOND, dict(total_q=1 << 48)),
    (FITS, dict(batch=1, heads_q=2, heads_kv=1, max_q=((1 << 24) - 1) * 16)), (BEYOND, dict(batch=1, heads_q=2, heads_kv=1, max_q=((1 << 24) - 1) * 16 + 1)),
    (BEYOND, dict(head_dim=264, q_head=264, k_head=264, v_head=264, o_head=264, **FAR)), (FITS, dict(head_dim=256, q_head=256, k_head=256, v_head=256, o_head=256, **FAR)),
], ids=str)
def test_attention(fake, want, change):  # noqa: F811
    t = 1 << 45
    places = {k: (1 << 44) + i * t for i, k in enumerate(("out", "lse", "q", "cu_q", "k_start", "k_len", "workspace", "k", "v"))}
    assert base.call_attn(fake, workspace_bytes=1 << 44, **{**places, **change}) == want


@pytest.mark.parametrize("want,change", [
    (FITS, dict(a_row=(1 << 23) - 16, b_row=(1 << 23) - 16)), (BEYOND, dict(a_row=1 << 23)), (BEYOND, dict(b_row=1 << 23)),
    (FITS, dict(rows=64 * 1023, cols=64 * 4100, out_row=64 * 4100)), (BEYOND, dict(rows=64 * 1024, cols=64 * 4096, out_row=64 * 4096)),
    (BEYOND, dict(rows=1 << 31)), (BEYOND, dict(out_row=1 << 31)), (FITS, dict(out_row=(1 << 31) - 1)),
], ids=str)
def test_matmul(fake, want, change):  # noqa: F811
    t = 1 << 44
    places = {k: (1 << 44) + i * t for i, k in enumerate(("out", "a", "a_scales", "b", "b_scales", "workspace"))}
    assert base.call_mm(fake, **{**places, **change}) == want


def test_quantize(fake):  # noqa: F811
    far = dict(codes=1 << 44, scales=1 << 45, x=1 << 46, rows=1)
    assert base.call_quant(fake, cols=(1 << 31) - 16, x_row=1 << 31, codes_row=1 << 31, **far) == FITS
    assert base.call_quant(fake, cols=1 << 31, x_row=1 << 31, codes_row=1 << 31, **far) == BEYOND
