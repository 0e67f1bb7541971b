"""GPU tests of the FP8 layer operators against their definitions in 64 bits
(tests/ops_ref.py), at the sizes, strides and masks where they can go wrong."""
import math

import pytest
import torch

from routed_moe_decode_router_gb300 import ops
from tests import ops_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_status() == 0


def randn(*shape, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    return torch.randn(*shape, generator=g, device="cuda") * std


def within(got, want, bound):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), "%d of %d, worst %.3g x its bound" % (
        int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / bound).max()))


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
# fp32 before the rounding: the sum of squares 30 steps (halved by the root),
# the root, the division and two products 6: under 32 U.

def check_norm(x, w, out, residual=None, eps=1e-6):
    t = x.dtype
    s, y = R.norm(x, w, eps, residual)
    if residual is not None:
        within(out.residual, s, s.abs() * (R.half_step(t) + 2 * R.U) + R.tiny_step(t))
    if out.y is not None:
        within(out.y, y, y.abs() * (R.half_step(t) + 33 * R.U) + R.tiny_step(t))
    if out.q is not None:
        k = x.shape[1]
        pad = torch.zeros(x.shape[0], -(-k // 128) * 128, dtype=torch.float64, device=x.device)
        pad[:, :k] = y.abs()
        sc = pad.unflatten(1, (-1, 128)).amax(2).clamp(min=1e-30) / 448.0
        within(out.scales, sc, sc * 34 * R.U)
        val = R.wide_rows(out.q, out.scales)
        within(val, y, y.abs() * (2.0 ** -4 + 72 * R.U) + R.expand_rows(sc, k) * 2.0 ** -10 * 1.001)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,hidden", [(1, 1), (1, 128), (3, 7), (2, 129), (9, 256), (5, 1000),
                                         (1, 4096), (33, 2048), (300, 2817), (3, 4104), (2, 9000),
                                         (2, 32768)])
def test_norm_sizes(dtype, rows, hidden):
    x, r = randn(rows, hidden).to(dtype), randn(rows, hidden, seed=1, std=3.0).to(dtype)
    w = (1 + randn(hidden, seed=2, std=0.1)).to(dtype)
    check_norm(x, w, ops.rms_norm(x, w, residual=r, quantize=True), r)
    out = ops.rms_norm(x, w, quantize=True, keep=False)
    assert out.y is None and out.residual is None
    check_norm(x, w, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("hidden", [264, 2048, 4096, 4100, 8192, 8200])
@pytest.mark.parametrize("rows", [152, 153])
def test_norm_at_a_row_for_every_sm_and_one_more(dtype, rows, hidden):
    x, r = randn(rows, hidden).to(dtype), randn(rows, hidden, seed=1, std=3.0).to(dtype)
    w = (1 + randn(hidden, seed=2, std=0.1)).to(dtype)
    check_norm(x, w, ops.rms_norm(x, w, residual=r, quantize=True), r)
    own = r.clone()
    check_norm(x, w, ops.rms_norm(x, w, residual=own, residual_out=own), r)


@pytest.mark.parametrize("offset", [0, 1, 8])
def test_norm_strided_rows_and_in_place(offset):
    big = randn(17, 600).to(torch.bfloat16)
    x, r = big[:, offset:offset + 264], big[:, 300 + offset:564 + offset]
    w = (1 + randn(264, seed=2, std=0.1)).to(torch.bfloat16)
    check_norm(x, w, ops.rms_norm(x, w, residual=r, quantize=True), r)
    own = r.contiguous()
    out = ops.rms_norm(x, w, residual=own, residual_out=own)
    assert out.residual.data_ptr() == own.data_ptr()
    check_norm(x, w, out, r)


def test_norm_rows_of_zeros_tiny_and_not_finite():
    x = randn(6, 384).to(torch.float32)
    x[0] = 0
    x[1, 128:256] = 0
    x[2] *= 1e-25
    x[3, 5] = math.nan
    x[4, 5] = math.inf
    w = torch.ones(384, device="cuda")
    out = ops.rms_norm(x, w, quantize=True, eps=0.0)
    assert out.y[0].isnan().all()            # 0 / 0 without an eps
    out = ops.rms_norm(x, w, quantize=True)
    assert not out.y[0].any() and not out.q[0].float().any()
    assert not out.q[1, 128:256].float().any() and out.scales.min() > 0
    assert out.y[3].isnan().all() and out.y[4, 5].isnan() and not out.y[4, :5].any()
    ok = [0, 1, 2, 5]
    check_norm(x[ok], w, ops.NormOut(out.y[ok], None, out.q[ok], out.scales[ok]))


def test_norm_no_rows():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    out = ops.rms_norm(x, torch.ones(256, dtype=torch.bfloat16, device="cuda"), quantize=True)
    assert out.y.shape == (0, 256) and out.scales.shape == (0, 2)


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------

def check_route(logits, top_k, **kw):
    ids, wts = ops.route_topk(logits, top_k, **kw)
    want_ids, want_w = R.route(logits, top_k, **kw)
    assert torch.equal(ids.cpu(), want_ids)
    e = logits.shape[1]
    # p: (e / 32 + 16) U, at most the same again from the renormalisation, then two products
    within(wts.cpu(), want_w, want_w.abs() * (2 * (e / 32 + 16) + 4) * R.U + 1e-37)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("rows,experts,top_k,groups,limit,score", [
    (1, 1, 1, 1, 1, "max"), (5, 16, 4, 1, 1, "max"), (7, 33, 33, 1, 1, "max"),
    (64, 160, 8, 1, 1, "max"), (33, 256, 8, 8, 4, "top2"), (33, 256, 8, 8, 4, "max"),
    (9, 120, 6, 3, 2, "top2"), (9, 96, 6, 32, 7, "top2"), (9, 32, 5, 32, 5, "top2"),
    (4, 512, 16, 4, 1, "top2"), (3, 1024, 64, 16, 16, "max"), (5, 700, 10, 7, 3, "top2")])
def test_route_sizes(scoring, bias, rows, experts, top_k, groups, limit, score):
    logits = randn(rows, experts, std=1.5)
    b = randn(experts, seed=3, std=0.1) if bias else None
    for norm, f in ((True, 2.5), (False, 1.0)):
        check_route(logits, top_k, scoring=scoring, bias=b, groups=groups, group_limit=limit,
                    group_score=score, norm_topk_prob=norm, routed_scaling_factor=f)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("scoring,bias", [("softmax", False), ("sigmoid", True)])
def test_route_ties_go_to_the_lower_index(dtype, scoring, bias):
    # few distinct values: most comparisons are ties, among groups too
    logits = (randn(40, 64) * 2).round().to(dtype) / 2
    logits[0] = 0.0
    logits[1, ::2], logits[1, 1::2] = 0.0, -0.0
    b = ((randn(64, seed=4) * 2).round() / 8) if bias else None
    for groups, limit in ((1, 1), (8, 3)):
        check_route(logits, 6, scoring=scoring, bias=b, groups=groups, group_limit=limit,
                    group_score="top2")


def test_route_decides_close_keys_as_in_64_bits():
    # keys one fp32 step or less apart: sigmoid saturates, the bias dominates
    logits = 20 + randn(50, 128)
    logits[:25] = 3 + randn(25, 128) * 1e-6
    b = torch.full((128,), 8.0, device="cuda")
    check_route(logits, 8, scoring="sigmoid", bias=b)
    check_route(logits, 8, scoring="sigmoid", bias=b, groups=8, group_limit=2, group_score="top2")
    check_route(logits, 8, scoring="softmax", bias=b)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top_k", [1, 8, 31, 32, 40])
def test_route_pairs_of_keys_a_step_apart(scoring, top_k):
    """Pairs of experts whose keys differ by about an fp32 step, in and at the
    end of the selection, more of them than lanes among them."""
    base = randn(30, 48, std=1.0).repeat_interleave(2, 1)
    logits = base + randn(30, 96, seed=1) * 1e-7
    logits[0] = logits[0, 0] + randn(96, seed=2) * 1e-7
    b = (randn(48, seed=3, std=0.1)).repeat_interleave(2)
    check_route(logits, top_k, scoring=scoring, bias=b, routed_scaling_factor=2.0)
    logits[1, 9:] = -math.inf
    logits[2, 3:] = -math.inf
    check_route(logits, top_k, scoring=scoring, bias=b, norm_topk_prob=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("score", ["max", "top2"])
@pytest.mark.parametrize("groups,limit", [(4, 1), (8, 3), (12, 11)])
def test_route_groups_a_step_apart(scoring, score, groups, limit):
    """Groups whose scores differ by about an fp32 step or not at all, with one
    to all of their experts behind the score."""
    size = 96 // groups
    one = randn(40, size, std=1.0)
    logits = one.repeat(1, groups) + randn(40, 96, seed=1) * 1e-7
    logits[10:20] = one[10:20].repeat(1, groups)
    logits[20:30] = randn(10, 96, seed=2) * 1e-7
    logits[30, size:] = -math.inf
    for bias in (None, randn(size, seed=3, std=0.1).repeat(groups)):
        check_route(logits, min(5, limit * size), scoring=scoring, bias=bias, groups=groups,
                    group_limit=limit, group_score=score)


@pytest.mark.parametrize("scoring,bias", [("softmax", False), ("softmax", True),
                                          ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("groups,limit", [(1, 1), (8, 2)])
def test_route_masked_experts(scoring, bias, groups, limit):
    logits = randn(12, 64)
    logits[0] = -math.inf                       # nothing is left
    logits[1, 3:] = -math.inf                   # fewer than top_k are left
    logits[2, ::2] = math.nan
    logits[3, 8:] = -math.inf                   # one group is left
    logits[4, [1, 9, 17]] = -math.inf
    logits[5] = torch.finfo(torch.float32).min  # the lowest value is a value
    logits[6] = -200.0                          # sigmoids too small for fp32
    logits[7, :] = torch.linspace(-300, 300, 64)
    b = randn(64, seed=5, std=0.1) if bias else None
    check_route(logits, 6, scoring=scoring, bias=b, groups=groups, group_limit=limit,
                group_score="top2")


def test_route_strided_rows_and_none():
    big = randn(10, 300)
    check_route(big[:, 7:135], 4)
    check_route(big[::3, 1:100].to(torch.float16)[:, 3:], 4, scoring="sigmoid")
    ids, wts = ops.route_topk(torch.empty(0, 64, device="cuda"), 4)
    assert ids.shape == wts.shape == (0, 4)


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------

def operands(m, n, k, seed=0):
    # scales that differ from block to block by orders of magnitude
    x = randn(m, k, seed=seed) * torch.exp(randn(m, -(-k // 128), seed=seed + 1)
                                           ).repeat_interleave(128, 1)[:, :k]
    w = randn(n, k, seed=seed + 2, std=0.02) * torch.exp(randn(-(-n // 128), 1, seed=seed + 3)
                                                         ).repeat_interleave(128, 0)[:n]
    return R.rows_fp8(x) + R.weights_fp8(w)


def check_product(a, sa, b, sb, got):
    want, mag = R.product(a, sa, b, sb)
    t = got.dtype
    e = mag * R.product_bound(a.shape[1])
    within(got, want, e + (want.abs() + e) * (R.half_step(t) if t != torch.float32 else 0)
           + R.tiny_step(t))


@pytest.mark.parametrize("m,n,k", [
    (1, 1, 16), (1, 128, 128), (128, 128, 128), (128, 256, 256), (5, 100, 144), (1, 4096, 4096),
    (33, 1000, 2048), (129, 257, 272), (200, 384, 1040), (64, 640, 8192), (127, 129, 128),
    (1000, 2000, 512), (300, 5000, 1152),
    (8, 1000, 1040), (9, 24, 4096), (16, 4096, 272), (17, 333, 2048), (32, 2048, 7168), (2, 40, 16),
    (31, 17, 16384)])
def test_matmul_sizes(m, n, k):
    a, sa, b, sb = operands(m, n, k)
    for t in (torch.float32, torch.bfloat16, torch.float16):
        check_product(a, sa, b, sb, ops.matmul_fp8(a, sa, b, sb, out_dtype=t))


def test_matmul_many_tiles_per_block():
    a, sa, b, sb = operands(2111, 2900, 640)
    check_product(a, sa, b, sb, ops.matmul_fp8(a, sa, b, sb, out_dtype=torch.float32))


def test_matmul_all_codes_and_wide_accumulation():
    """Every finite code, and a product whose blocks cancel to the last bits."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    codes = codes[(codes & 0x7F) != 0x7F]
    a = codes.repeat(129)[:128 * 254].view(128, 254)[:, :240].contiguous().view(ops.F8)
    b = codes.flip(0).repeat(130)[:130 * 240].view(130, 240).contiguous().view(ops.F8)
    sa, sb = randn(128, 2).abs() + 0.1, randn(2, 2, seed=1).abs() + 0.1
    check_product(a, sa, b, sb, ops.matmul_fp8(a, sa, b, sb, out_dtype=torch.float32))
    one = torch.ones(4, 256, device="cuda").to(ops.F8)
    s = torch.tensor([[1.0, -1.0]] * 4, device="cuda")
    w = torch.ones(8, 256, device="cuda").to(ops.F8)
    out = ops.matmul_fp8(one, s, w, torch.ones(1, 2, device="cuda"), out_dtype=torch.float32)
    assert not out.any()


@pytest.mark.parametrize("n", [130, 131, 133, 260, 257, 271, 383, 388, 519])
@pytest.mark.parametrize("offset", [0, 1, 2, 4])
def test_matmul_rows_of_outputs_at_every_alignment(n, offset):
    a, sa, b, sb = operands(150, n, 256)
    for t in (torch.bfloat16, torch.float32):
        flat = torch.full((150 * n + 16,), 77.0, dtype=t, device="cuda")
        out = flat[offset:offset + 150 * n].view(150, n)
        ops.matmul_fp8(a, sa, b, sb, out=out)
        check_product(a, sa, b, sb, out)
        assert (flat[:offset] == 77).all() and (flat[offset + 150 * n:] == 77).all()


def test_matmul_strided_operands_and_given_output():
    a, sa, b, sb = operands(70, 200, 640)
    wa = torch.zeros(70, 1024, dtype=torch.uint8, device="cuda").view(ops.F8)
    wb = torch.zeros(200, 656, dtype=torch.uint8, device="cuda").view(ops.F8)
    va, vb = wa[:, 16:656], wb[:, :640]
    va.view(torch.uint8).copy_(a.view(torch.uint8))
    vb.view(torch.uint8).copy_(b.view(torch.uint8))
    out = torch.full((70, 200), math.nan, device="cuda")
    ops.matmul_fp8(va, sa, vb, sb, out=out)
    check_product(a, sa, b, sb, out)
    assert torch.equal(out, ops.matmul_fp8(a, sa, b, sb, out_dtype=torch.float32))
    # an output whose rows start on odd elements
    odd = torch.full((70 * 200 + 3,), math.nan, dtype=torch.bfloat16, device="cuda")
    view = odd[1:-2].view(70, 200)
    ops.matmul_fp8(a, sa, b, sb, out=view)
    check_product(a, sa, b, sb, view)
    assert odd[0].isnan() and odd[-2:].isnan().all()


def test_matmul_codes_that_are_no_number_stay_in_their_row():
    a, sa, b, sb = operands(40, 300, 256)
    a.view(torch.uint8)[7, 100] = 0x7F
    out = ops.matmul_fp8(a, sa, b, sb)
    assert out[7].isnan().all()
    keep = [i for i in range(40) if i != 7]
    check_product(a[keep], sa[keep], b, sb, out[keep])


def test_matmul_no_rows():
    a, sa, b, sb = operands(3, 128, 256)
    assert ops.matmul_fp8(a[:0], sa[:0], b, sb).shape == (0, 128)


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------

def layer(e, h, i, seed=0):
    def stack(n, k, s):
        qs = [R.weights_fp8(randn(n, k, seed=s + 7 * j, std=0.05)) for j in range(e)]
        return torch.stack([q.view(torch.uint8) for q, _ in qs]).view(ops.F8), torch.stack(
            [s for _, s in qs])
    return stack(i, h, seed) + stack(i, h, seed + 1) + stack(h, i, seed + 2)


def choice(t, k, e, seed=0, std=1.0):
    """Some experts are asked far more often than others."""
    p = randn(t, e, seed=seed) + randn(e, seed=seed + 1, std=std)
    w, ids = p.softmax(1).topk(k, dim=1)
    return ids.to(torch.int32), w.contiguous()


def check_experts(x, ids, wts, lay, **kw):
    q, s = R.rows_fp8(x)
    got = ops.experts_fp8(q, s, ids, wts, *lay, **kw)
    want, bound = R.experts(q, s, ids, wts, *lay, addend=kw.get("addend"))
    within(got, want, bound)
    return got


@pytest.mark.parametrize("t,e,k,h,i", [
    (1, 1, 1, 128, 128), (1, 16, 4, 256, 128), (3, 8, 8, 384, 256), (7, 16, 2, 2048, 768),
    (40, 3, 2, 256, 384), (130, 4, 4, 512, 128), (300, 1, 1, 640, 256), (257, 37, 6, 384, 640),
    (64, 64, 8, 1024, 256), (1000, 16, 4, 256, 256), (2, 1024, 64, 128, 128), (4, 40, 8, 512, 384),
    (33, 5, 1, 256, 256), (32, 1, 1, 512, 256), (8, 64, 4, 4096, 1536), (16, 2, 2, 256, 2048),
    (1, 64, 32, 256, 128), (4, 1000, 8, 128, 4096)])
def test_experts_sizes(t, e, k, h, i):
    ids, wts = choice(t, k, e)
    check_experts(randn(t, h, seed=9), ids, wts, layer(e, h, i))


@pytest.mark.parametrize("t", [1, 2, 7, 40])
def test_experts_few_rows_each_over_and_over(t):
    """Tiles of one to a few rows with long inputs: the loading warps have
    unequal shares and must not lose each other."""
    lay = layer(64, 2048, 128)
    ids, wts = choice(t, 8, 64, std=0.1)
    x = randn(t, 2048, seed=9)
    first = check_experts(x, ids, wts, lay)
    q, s = R.rows_fp8(x)
    for _ in range(200):
        again = ops.experts_fp8(q, s, ids, wts, *lay)
    assert torch.equal(first, again) and ops.device_status() == 0


def test_experts_index_in_a_cluster():
    """More pairs than one block sorts, one expert with most of them."""
    ids, wts = choice(1500, 4, 8, std=3.0)
    check_experts(randn(1500, 128, seed=9), ids, wts, layer(8, 128, 128))


def test_experts_slots_without_an_expert():
    lay = layer(6, 256, 256)
    ids, wts = choice(50, 4, 6)
    ids[3] = -1
    ids[5, 1:] = -1
    ids[7, 0], ids[8, 3] = 6, 1 << 30
    ids[9, 2] = -(1 << 31)
    got = check_experts(randn(50, 256, seed=9), ids, wts, lay)
    assert not got[3].any()
    ids[:] = -1
    assert not check_experts(randn(50, 256, seed=9), ids, wts, lay).any()


def test_experts_repeated_ids_and_one_expert_for_all():
    lay = layer(4, 256, 128)
    ids = torch.full((150, 3), 2, dtype=torch.int32, device="cuda")
    check_experts(randn(150, 256, seed=9), ids, randn(150, 3).abs(), lay)


@pytest.mark.parametrize("t,k", [(1, 1), (4, 8), (10, 3), (32, 1), (40, 2)])
def test_experts_few_pairs_dropped_and_repeated(t, k):
    lay = layer(5, 384, 256)
    g = torch.Generator(device="cuda").manual_seed(t)
    ids = torch.randint(-2, 7, (t, k), generator=g, device="cuda").to(torch.int32)
    ids[t // 2] = 3
    add = randn(t, 384, seed=12).to(torch.bfloat16)
    check_experts(randn(t, 384, seed=9), ids, randn(t, k, seed=10), lay, addend=add)
    got = check_experts(randn(t, 384, seed=9), torch.full_like(ids, 5), randn(t, k), lay)
    assert not got.any()


def test_experts_addend_output_and_workspace():
    lay = layer(8, 256, 128)
    ids, wts = choice(20, 2, 8)
    add = randn(20, 256, seed=11).to(torch.bfloat16)
    ws = ops.ExpertsWorkspace(64, 2, 256, 128, 8)
    x = randn(20, 256, seed=9)
    a = check_experts(x, ids, wts, lay, addend=add, ws=ws)
    out = add.clone()
    q, s = R.rows_fp8(x)
    assert ops.experts_fp8(q, s, ids, wts, *lay, ws=ws, addend=out, out=out) is out
    assert torch.equal(a, out)
    ws.buf.fill_(0xFF)       # needs no initialisation
    assert torch.equal(a, check_experts(x, ids, wts, lay, addend=add, ws=ws))


def test_experts_rows_do_not_depend_on_their_neighbours():
    lay = layer(16, 512, 256)
    ids, wts = choice(200, 4, 16)
    q, s = R.rows_fp8(randn(200, 512, seed=9))
    whole = ops.experts_fp8(q, s, ids, wts, *lay)
    assert torch.equal(whole, ops.experts_fp8(q, s, ids, wts, *lay))
    # a smaller call may split the inputs differently; its rows agree to the last rounding
    part = ops.experts_fp8(q[:100], s[:100], ids[:100].contiguous(), wts[:100].contiguous(), *lay)
    want, bound = R.experts(q, s, ids, wts, *lay)
    within(part, want[:100], bound[:100])


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------

def test_all_on_another_stream_and_in_a_graph():
    lay = layer(8, 256, 128)
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    x, r = randn(9, 256).to(torch.bfloat16), randn(9, 256, seed=1).to(torch.bfloat16)
    proj = R.weights_fp8(randn(8, 256, seed=2, std=0.1))
    ws = ops.ExpertsWorkspace(9, 2, 256, 128, 8)

    def path(stream=None):
        n = ops.rms_norm(x, w, residual=r, quantize=True, stream=stream)
        logits = ops.matmul_fp8(n.q, n.scales, *proj, out_dtype=torch.float32, stream=stream)
        ids, wts = ops.route_topk(logits, 2, stream=stream)
        out = ops.experts_fp8(n.q, n.scales, ids, wts, *lay, ws=ws, addend=n.residual,
                              stream=stream)
        if stream is not None:
            stream.synchronize()
        return out
    want = path().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(path(), want)
    torch.cuda.synchronize()
    assert torch.equal(path(stream=side), want)
    n = ops.rms_norm(x, w, quantize=True, stream=side)
    ids = torch.zeros(9, 1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    got = ops.experts_fp8(n.q, n.scales, ids, ids.float() + 1, *lay, stream=side)
    side.synchronize()
    assert torch.equal(got, ops.experts_fp8(n.q, n.scales, ids, ids.float() + 1, *lay))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = path()
    for seed in (20, 21):
        x.copy_(randn(9, 256, seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, path())


def test_refusals_with_device_tensors():
    a, sa, b, sb = operands(4, 128, 256)
    ids, wts = choice(4, 2, 8)
    lay = layer(8, 256, 128)
    for call, text in (
            (lambda: ops.matmul_fp8(a, sa.double(), b, sb), "dtype"),
            (lambda: ops.matmul_fp8(a, sa[:, :1], b, sb), "shape"),
            (lambda: ops.matmul_fp8(a, sa, b.t(), sb), "shape|contiguous"),
            (lambda: ops.matmul_fp8(a, sa, b, sb.cpu()), "is on"),
            (lambda: ops.matmul_fp8(a, sa, b, sb, out_dtype=torch.int32), "out_dtype"),
            (lambda: ops.route_topk(sa, 2, scoring="none"), "scoring"),
            (lambda: ops.route_topk(sa, 2, group_score="sum"), "group_score"),
            (lambda: ops.rms_norm(sa, sa[0].half()), "dtype"),
            (lambda: ops.rms_norm(sa, sa[0], residual_out=sa), "without residual"),
            (lambda: ops.rms_norm(sa, sa[0], keep=False), "no output"),
            (lambda: ops.experts_fp8(a, sa, ids.long(), wts, *lay), "dtype"),
            (lambda: ops.experts_fp8(a, sa, ids, wts.t(), *lay), "shape")):
        with pytest.raises(ValueError, match=text):
            call()
    from routed_moe_decode_router_gb300 import native as N
    with pytest.raises(N.MoeError, match="top_k"):
        ops.route_topk(sa, 3)
    with pytest.raises(N.MoeError, match="needs"):
        ops.experts_fp8(a, sa, ids, wts, *lay, ws=ops.ExpertsWorkspace(1, 2, 256, 128, 8))


@pytest.mark.parametrize("rows", [1, 5, 70])
@pytest.mark.parametrize("scoring,groups,limit", [("softmax", 1, 1), ("sigmoid", 4, 2)])
def test_layer_of_all_operators(rows, scoring, groups, limit):
    """The layer's steps against the definitions, each on what the step before
    it gave, and its output byte for byte."""
    from routed_moe_decode_router_gb300 import fp8_layer
    lay = fp8_layer.random_layer(512, 16, 256, 4, seed=3, shared_inter=384, scoring=scoring,
                                 groups=groups, group_limit=limit, group_score="top2")
    x, r = randn(rows, 512).to(torch.bfloat16), randn(rows, 512, seed=1).to(torch.bfloat16)
    out, res = lay.forward(x, r)
    n = ops.rms_norm(x, lay.norm, residual=r, quantize=True)
    check_norm(x, lay.norm, n, r)
    assert torch.equal(res, n.residual)
    logits = ops.matmul_fp8(n.q, n.scales, *lay.router, out_dtype=torch.float32)
    check_product(n.q, n.scales, *lay.router, logits)
    kw = dict(scoring=scoring, bias=lay.bias, groups=groups, group_limit=limit,
              group_score="top2")
    check_route(logits[:, :16].contiguous(), 4, **kw)
    ids, wts = ops.route_topk(logits[:, :16], 4, **kw)
    gate = torch.sigmoid(logits[:, 16:].double())
    shared, sb = R.experts(n.q, n.scales, torch.zeros_like(ids[:, :1]), gate, *lay.shared)
    want, bound = R.experts(n.q, n.scales, ids, wts, *lay.routed)
    # the shared output is rounded once more on its way; the gate within 8 U
    total = bound + sb + shared.abs() * (R.half_step(torch.bfloat16) + 8 * R.U)
    total = total + (want + shared).abs() * R.half_step(torch.bfloat16)
    within(out, want + shared, total)
    again, _ = lay.forward(x, r)
    assert torch.equal(again, out)
    first, res = lay.forward(x)
    assert res is x and first.shape == x.shape


def test_layer_weights_quantised_by_blocks():
    from routed_moe_decode_router_gb300 import fp8_layer
    w = randn(2, 200, 300) * torch.exp(randn(2, 200, 1, seed=1))
    q = fp8_layer.quantize_weights(w)
    for i in range(2):
        c, s = R.weights_fp8(w[i])
        assert torch.equal(s, q.scales[i])
        assert (R.wide_weights(q.codes[i], q.scales[i]) - w[i].double()).abs().max() <= \
            2.0 ** -4 * w[i].abs().max()
