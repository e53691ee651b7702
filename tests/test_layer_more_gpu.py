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


# ------------------------------------------------------------------ products of many blocks

def codes(rows, depth, pad, g):
    """e4m3 rows `pad` codes apart, which are NaN."""
    c = (torch.randn(rows, depth + pad, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    c.view(torch.uint8)[:, depth:] = 0x7F
    return c[:, :depth]


def block_scales(rows, blocks, g):
    """From 2^-8 to 1, other powers of two from each block to the next."""
    power = (torch.arange(blocks) * 5 + torch.arange(rows)[:, None] * 3) % 9 - 8
    return (0.5 + 0.5 * torch.rand(rows, blocks, generator=g)) * 2.0 ** power


MANY = [  # rows and columns: 256 x 256 tiles (128 x 128 in binary32), 128 x 256, 128 x 128; depth of 17, 18, 25 and 34 blocks
    (2100, 4100, 2064), (2100, 4100, 4240), (2304, 4096, 3200), (1400, 4000, 2064), (1400, 4000, 2192), (1408, 4096, 4240),
    (900, 4000, 2064), (900, 4000, 4240), (896, 4096, 3200),
]


@pytest.mark.parametrize("kind", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("m,n,k", MANY)
def test_matmul_of_many_blocks(ctx, m, n, k, kind):
    """Scales come eight blocks at a time through two buffers: from the third eight on each is in use again.

    Beside each element's bound, the errors' root mean square over sampled rows: a rounding to the type is off
    by its half step at the value over sqrt 3 at most, a block's inner sum in a 16-bit result by 1.45e-5 of the
    products' root sum of squares (normal values; measured on the instruction itself), 2^-15 with a margin
    of two, in a binary32 one by the root of 128 half steps of it, and each of the additions by half a step."""
    log_case(f"many blocks {m} x {n} x {k} {kind}")
    g, kb = base.gen(m + k), -(-k // 128)
    a, b = codes(m, k, 16, g), codes(n, k, 48, g)
    sa, sb = block_scales(m, kb, g), block_scales(-(-n // 128), kb, g) * 2.0 ** -8
    pad = 0 if n % 8 == 0 else 3
    out = torch.full((m + 1, n + pad), 7.0, dtype=kind, device="cuda")
    ar.ar_fp8_matmul(ctx, out[:m, :n], _device_rows(a), sa.cuda(), _device_rows(b), sb.cuda())
    torch.cuda.synchronize()
    rows = torch.cat([torch.arange(0, m, 83), torch.tensor([m - 2, m - 1])])
    want, tol = ref.matmul(a[rows], sa[rows], b, sb, kind)
    got = out.cpu()
    base.near(got[rows, :n], want, tol, "product")
    assert bool((got[m] == 7).all()) and bool((got[:, n:] == 7).all())
    rss, mass = torch.zeros_like(want), torch.zeros_like(want)
    for c in range(kb):
        x, y = a[rows][:, 128 * c:128 * c + 128].double(), b[:, 128 * c:128 * c + 128].double()
        f = sa[rows, c].double()[:, None] * sb[:, c].double().repeat_interleave(128)[:n][None]
        rss += (f * f) * (x.square() @ y.square().t())
        mass += f * (x @ y.t()).abs()
    inner = 2.0 ** -15 if kind != F32 else (128 ** 0.5) * ref.U32
    most = ref.U[kind] ** 2 / 3 * want.square().mean() + inner ** 2 * rss.mean() + (3 * ref.U32) ** 2 * mass.square().mean()
    seen = (got[rows, :n].double() - want).square().mean()
    print(f"rms {float(seen.sqrt()):.3e} of {float(most.sqrt()):.3e}")
    assert float(seen) <= float(most)


def _device_rows(x):
    """The same rows at the same pitch on the device (what lies between them too)."""
    whole = torch.as_strided(x, (x.shape[0], x.stride(0)), (x.stride(0), 1))
    return whole.cuda()[:, :x.shape[1]]


# ------------------------------------------------------------------ calls past one launch, offsets past 32 bits

def need_memory(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB")


def test_qk_past_one_launch(ctx):
    """2^24 + 5 tokens of one query and one key head of 504: 2^31 lanes and more, queries past 2^32 elements, in place."""
    need_memory(60)
    log_case("norm and rotation past one launch")
    t, d = (1 << 24) + 5, 504
    q, k = (torch.empty(t, 1, d, dtype=BF16, device="cuda").normal_() for _ in range(2))
    rows = torch.tensor([0, 1, 8388607, 8388608, (1 << 24) - 1, 1 << 24, (1 << 24) + 4])
    table, w = ref.rope_table(50, 8), torch.randn(2, d, generator=base.gen(1)).to(BF16)
    pos = torch.arange(t, device="cuda") % 50
    slots = torch.full((t,), -1, dtype=torch.int64, device="cuda")
    slots[rows.cuda()] = torch.arange(len(rows), device="cuda") * 2
    hq, hk = q[rows.cuda()].cpu(), k[rows.cuda()].cpu()
    cache = torch.full((2 * len(rows), 1, d), 7.0, dtype=BF16, device="cuda")
    ar.ar_qk_norm_rope(ctx, q, k, w[0].contiguous().cuda(), w[1].contiguous().cuda(), table.cuda(), pos, k_out=cache, slots=slots, eps=1e-5)
    torch.cuda.synchronize()
    at = rows % 50
    base.near(q[rows.cuda()], *ref.qk(hq, w[0], table, at, 1e-5, False), "q")
    base.near(cache[0::2], *ref.qk(hk, w[1], table, at, 1e-5, False), "keys")
    assert bool((cache[1::2] == 7).all()) and torch.equal(k[rows.cuda()].cpu(), hk)


def test_quantize_past_one_launch(ctx):
    """2^28 + 300 rows of 16: 2^31 lanes and more, past 2^32 elements."""
    need_memory(40)
    log_case("codes past one launch")
    r = (1 << 28) + 300
    x = torch.empty(r, 16, dtype=BF16, device="cuda").normal_()
    out, scales = torch.empty(r, 16, dtype=torch.uint8, device="cuda"), torch.empty(r, 1, device="cuda")
    ar.ar_fp8_quantize(ctx, out, scales, x)
    torch.cuda.synchronize()
    rows = torch.cat([torch.arange(100), torch.arange((1 << 28) - 100, r)])
    want, want_s = ref.quantize(x[rows.cuda()].cpu())
    assert torch.equal(scales[rows.cuda()].cpu(), want_s)
    base.same_bytes(out[rows.cuda()], want, "codes")


def test_matmul_past_32_bits(ctx):
    """A result of 4.9e9 elements."""
    need_memory(24)
    log_case("product past 32 bits")
    m = n = 70000
    g = base.gen(7)
    a, b = codes(m, 128, 0, g), codes(n, 128, 0, g)
    sa, sb = torch.rand(m, 1, generator=g) * 1e-3, torch.rand(-(-n // 128), 1, generator=g)
    out = torch.empty(m, n, dtype=BF16, device="cuda")
    ar.ar_fp8_matmul(ctx, out, a.cuda(), sa.cuda(), b.cuda(), sb.cuda())
    torch.cuda.synchronize()
    rows = torch.tensor([0, 30678, 30679, 61356, 61357, 69998, 69999])      # 2^31 and 2^32 elements lie between the middle ones
    want, tol = ref.matmul(a[rows], sa[rows], b, sb, BF16)
    base.near(out[rows.cuda()], want, tol, "product")


@pytest.mark.parametrize("lens_q", [[1100], [1] * 1100], ids=["a prompt", "single tokens"])
def test_attention_of_queries_past_32_bits(ctx, lens_q):
    """Queries and results 2^22 elements apart."""
    need_memory(24)
    log_case(f"queries past 32 bits, {len(lens_q)} sequences")
    q, k, v, cu, ks, kl = base.attn_case(BF16, lens_q, [70] * len(lens_q), 4, 2, 64)
    wide = torch.empty(2, q.shape[0], 1 << 22, dtype=BF16, device="cuda")
    dq, out = (wide[i][:, -256:].view(-1, 4, 64) for i in range(2))
    dq.copy_(q)
    lse = torch.empty(q.shape[:2], device="cuda")
    ar.ar_attention(ctx, out, dq, k.cuda(), v.cuda(), cu.cuda(), ks.cuda(), kl.cuda(), max(lens_q), 70, lse=lse)
    torch.cuda.synchronize()
    used = int(cu[-1])
    want, wl, tol, tl = ref.attention(q, k, v, cu, ks, kl, True, 64 ** -0.5)
    base.near(out[:used], want[:used], tol[:used], "far queries")
    base.near(lse[:used], wl[:used], tl[:used], "their lse")


# ------------------------------------------------------------------ codes by what they stand for

@pytest.mark.parametrize("kind", [BF16, F16, F32], ids=str)
def test_codes_stand_for_their_elements(ctx, kind):
    """Scale times code against the element itself: half a step of e4m3, 2^-4 of the value, or of its
    smallest ones, 2^-10; and the few binary32 roundings of the factor, the product and the scale."""
    log_case(f"codes stand for their elements {kind}")
    x = torch.randn(300, 1040, generator=base.gen(4)) * torch.logspace(-6, 4, 300, base=2.0)[:, None]
    x[::7, 5::50] *= 100
    x = x.to(kind)
    out, scales = torch.empty(300, 1040, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(300, 9, device="cuda")
    ar.ar_fp8_quantize(ctx, out, scales, x.cuda())
    torch.cuda.synchronize()
    s = scales.cpu().double().repeat_interleave(128, 1)[:, :1040]
    top = torch.stack([x[:, c:c + 128].double().abs().amax(1) for c in range(0, 1040, 128)], 1) / 448
    base.near(scales, top, ref.U32 * top, "scales")
    want = x.double() / s
    base.near(out.float(), want, 2.0 ** -4 * want.abs() + 2.0 ** -10 + 6 * ref.U32 * want.abs(), "codes")
