"""The FP8 decode for more than 16 query rows per latent head (mla_decode_paged_fp8_rows)
against the decode written out in fp64.

Tolerances, element by element: half a bf16 step of the output (2^-8); the two 8-bit terms of
v = P s; and the query's, whose part in a score of size x is at most 2^-18 * max|q| * sum|k| * scale
(below 3e-4 for the drawn inputs) and moves every probability by that much.  The terms of v: for v
in [2^k, 2^(k+1)) the nearest E4M3 value (steps of 2^(k-3)) leaves at most 2^(k-4); E5M2 below
2^(k-4) has steps of at most 2^(k-7), so the rest is kept within 2^(k-8) <= 2^-8 v.  That holds for
v >= 2^-6; below, E4M3's steps stay at 2^-9, the rest is at most 2^-10 and kept within 2^-14.  With
v = P s 2^(6-e), 2^e <= 2 max(s) and P = 1 for a probability of at most the row's largest, v < 2^-6
means p s < 2^-11 max(p) max(s), and 2^-14 is 2^-19 max(p) max(s).  Together at most
(2^-8 + 1e-3) * sum_j p_j |c_j| + 2^-19 max(p) max(s) * (sum of |code_j| over those small ones).
LSE: the library's 1e-4 of max(|lse|, 1)."""

import math

import pytest
import torch

from paged_mla_decode_11_b200 import ops
from paged_mla_decode_11_b200 import workloads as W

pytestmark = pytest.mark.gpu


def reference(x):
    """(out, the error its terms may have, lse) in fp64."""
    q, h, g = x["q"].cuda().double(), x["h_kv"], x["h_q"] // x["h_kv"]
    b, s_q, h_q, _ = q.shape
    out = torch.zeros(b, s_q, h_q, 512, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(out)
    lse = torch.full((b, h_q, s_q), -torch.inf, dtype=torch.float64, device="cuda")
    k8, ks = x["k8"].cuda().view(torch.uint8), x["k_scale"].cuda()
    for i, L in enumerate(x["cache_seqlens"].tolist()):
        if L == 0:
            continue
        pages = x["block_table"][i, :-(-L // 64)].long().cuda()
        c = k8[pages].view(torch.float8_e4m3fn).float().double() * ks[:, pages].permute(1, 2, 0)[..., None].double()
        c = c.flatten(0, 1)[:L]
        for n in range(h):
            rows = q[i, :, n * g:(n + 1) * g] @ c[:, n].t() * x["softmax_scale"]      # [s_q, g, L]
            if x["causal"]:
                keep = torch.arange(L, device="cuda") < L - (s_q - 1 - torch.arange(s_q, device="cuda"))[:, None]
                rows = rows.masked_fill(~keep[:, None], -torch.inf)
            z = torch.logsumexp(rows, -1)
            p = torch.where(z[..., None] == -torch.inf, 0.0, (rows - z[..., None]).exp())
            out[i, :, n * g:(n + 1) * g] = p @ c[:, n, :512]
            s, top = ks[n, pages].flatten()[:L].double(), p.amax(-1, keepdim=True)
            small = (p * s < 2.0 ** -11 * top * s.max()).double()
            codes = k8[pages, :, n].view(torch.float8_e4m3fn).float().double().flatten(0, 1)[:L, :512].abs()
            size[i, :, n * g:(n + 1) * g] = (2.0 ** -8 + 1e-3) * (p @ c[:, n, :512].abs()) + \
                2.0 ** -19 * top * s.max() * (small @ codes)
            lse[i, n * g:(n + 1) * g] = z.t()
    return out, size, lse


def run(x, num_parts=None, **kw):
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    R = x["s_q"] * x["h_q"] // x["h_kv"]
    tile, splits = ops.get_mla_metadata(d["cache_seqlens"], R, x["h_kv"], num_parts=num_parts)
    b, s_q, h_q, _ = d["q"].shape
    ws = ops.new_workspace(ops.workspace_size(b, s_q, h_q, x["h_kv"], tile.shape[0]), "cuda")
    out, lse = ops.mla_decode_paged_fp8_rows(d["q"], d["k8"], d["k_scale"], d["block_table"], d["cache_seqlens"], 512,
                                             tile, splits, softmax_scale=x["softmax_scale"], causal=x["causal"],
                                             workspace=ws, **kw)
    torch.cuda.synchronize()
    assert ops.query_status(ws) == ops.MLA_OK, "a device-side wait timed out"
    return out, lse, (tile, splits, ws)


def parity(x, num_parts=None):
    out, lse, _ = run(x, num_parts)
    ref, size, ref_lse = reference(x)
    gone = ref_lse == -torch.inf
    assert torch.equal(lse == -torch.inf, gone)
    assert (out[gone.transpose(1, 2)] == 0).all()
    err = (lse.double() - ref_lse).abs()[~gone] / ref_lse.abs().clamp_min(1)[~gone]
    assert not err.numel() or err.max() <= 1e-4, f"lse off by {err.max():.3e}"
    tol = 2.0 ** -8 * ref.abs() + size + 1e-30
    worst = ((out.double() - ref).abs() / tol).max()
    assert worst <= 1, f"out off by {worst:.3f} of the tolerance"
    return float(worst), float(err.max()) if err.numel() else 0.0


CASES = [
    # (batch, s_q, h_q, h_kv, seqlens, causal)
    (1, 1, 128, 1, [1], False),                       # one key
    (2, 1, 128, 1, [37, 130], True),
    (5, 1, 128, 1, [1, 63, 64, 65, 300], False),      # ragged ends around pages
    (4, 1, 128, 1, [128, 129, 191, 192], True),       # one page, two pages, a lone third
    (3, 1, 128, 1, [0, 5, 0], True),                  # empty sequences
    (3, 1, 17, 1, [200, 1, 70], True),                # the fewest rows of this kernel
    (2, 1, 24, 1, [500, 77], True),
    (2, 1, 64, 1, [700, 130], False),                 # half a row block
    (2, 1, 100, 1, [333, 64], True),
    (2, 2, 64, 1, [1, 66], True),                     # causal, a row with no visible key
    (2, 4, 128, 1, [3, 700], True),                   # four blocks of rows, rows without keys
    (2, 3, 40, 1, [129, 65], True),                   # 120 rows, positions across a block
    (2, 2, 96, 1, [257, 1000], True),                 # 192 rows: one and a half blocks
    (2, 1, 64, 2, [500, 77], True),                   # two latent heads, 32 rows each
    (2, 2, 256, 2, [300, 65], False),
    (1, 1, 128, 1, [20000], False),                   # one long sequence over many parts
    (40, 1, 128, 1, list(range(1, 400, 10)), True),   # many short pieces per part
]


@pytest.mark.parametrize("b,s_q,h_q,h_kv,lens,causal", CASES)
def test_parity(b, s_q, h_q, h_kv, lens, causal):
    x = W.make_inputs_fp8(W.custom(b, s_q, h_q, h_kv, lens, causal=causal, outlier_frac=0.05), seed=sum(lens) + h_q)
    parity(x)


@pytest.mark.parametrize("num_parts", [1, 2, 5, 37])
def test_part_counts(num_parts):
    # few parts walk many pieces, one after another, through the rings; more split the sequences
    x = W.make_inputs_fp8(W.custom(9, 1, 128, 1, [5, 700, 64, 0, 129, 1, 1500, 63, 300], causal=True), seed=num_parts)
    parity(x, num_parts=num_parts)


def test_up_to_16_rows_is_the_other_call():
    x = W.make_inputs_fp8(W.custom(3, 1, 16, 1, [300, 1, 70], causal=True), seed=3)
    out, lse, (tile, splits, _) = run(x)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    o2, l2 = ops.mla_decode_paged_fp8(d["q"], d["k8"], d["k_scale"], d["block_table"], d["cache_seqlens"], 512, tile,
                                      splits, softmax_scale=x["softmax_scale"], causal=True)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("q_exp", [40, -40, 0])
def test_query_magnitudes(q_exp):
    # the query is carried per row, so rows far apart in size and far from one keep their accuracy
    x = W.make_inputs_fp8(W.custom(2, 1, 128, 1, [700, 130], causal=True), seed=17)
    q = x["q"].float() * 2.0 ** q_exp
    q[:, :, 3] = q[:, :, 3] * 2.0 ** -30                  # nearly uniform probabilities
    q[:, :, 70] = 0                                       # uniform ones
    x["q"] = q.to(torch.bfloat16)
    x["softmax_scale"] = 576 ** -0.5 * 2.0 ** -q_exp
    parity(x)


def test_scales_of_many_sizes():
    x = W.make_inputs(W.custom(3, 1, 128, 1, [1000, 640, 129], causal=False), seed=31)
    g = torch.Generator().manual_seed(31)
    k8 = torch.randint(0, 256, x["k_cache"].shape, generator=g, dtype=torch.int32).to(torch.uint8)
    k8[(k8 & 0x7f) == 0x7f] = 0x01                       # no NaN codes
    sub = torch.rand(k8.shape, generator=g) < 0.3
    k8[sub] = k8[sub] & 0x87                              # subnormals
    x["k8"] = k8
    # within a page by 2^6, from page to page by 2^12, growing and falling along a sequence
    page = torch.randint(-12, 1, (1, k8.shape[0], 1), generator=g)
    x["k_scale"] = (2.0 ** (page + torch.randint(-9, -2, (1, k8.shape[0], 64), generator=g))).float()
    x["k_scale"][0, x["block_table"][1, 3], 7] = 0.0
    parity(x)


def test_growing_scores():
    # the running maximum and the scales grow along the sequence, so the output is rescaled often
    x = W.make_inputs(W.custom(1, 1, 128, 1, [3000], causal=False), seed=5)
    L = 3000
    kc = x["k_cache"].float()
    order = x["block_table"][0, :47].long()
    for i, pg in enumerate(order.tolist()):
        kc[pg] *= 0.05 * 1.12 ** i
    x["k_cache"] = kc.to(torch.bfloat16)
    x["k8"], x["k_scale"] = W.to_fp8_cache(x["k_cache"])
    parity(x, num_parts=1)


def test_tails_and_foreign_rows():
    # scales of the slots past a sequence's end may be anything; a row with a NaN query stays alone
    x = W.make_inputs_fp8(W.custom(4, 1, 128, 1, [37, 130, 69, 64], causal=True), seed=17)
    out, lse, _ = run(x)
    y = dict(x, k_scale=x["k_scale"].clone(), q=x["q"].clone())
    for b, L in enumerate(x["cache_seqlens"].tolist()):
        if L % 64:
            page = int(x["block_table"][b, (L - 1) // 64])
            y["k_scale"][:, page, L % 64:] = float("nan") if b % 2 == 0 else float("inf")
    y["q"][1, 0, 5, 100] = float("nan")
    y["q"][2, 0, 127, 575] = float("inf")
    out2, lse2, _ = run(y)
    bad = torch.zeros(4, 1, 128, dtype=torch.bool, device="cuda")
    bad[1, 0, 5] = bad[2, 0, 127] = True
    assert torch.equal(out2[~bad], out[~bad]) and torch.equal(lse2[~bad.transpose(1, 2)], lse[~bad.transpose(1, 2)])
    assert torch.isnan(out2[bad]).all() and torch.isnan(lse2[bad.transpose(1, 2)]).all()


def test_strided_query_separate_combine_and_repeats():
    x = W.make_inputs_fp8(W.custom(2, 2, 128, 1, [5000, 300], causal=True), seed=9)
    out, lse, (tile, splits, _) = run(x)
    assert int(splits[1] - splits[0]) > 1
    out_b, lse_b, (_, _, ws) = run(x, skip_combine=True)
    ops.mla_combine(splits, 2, 128, 1, tile.shape[0], ws, out_b, lse_b)
    assert torch.equal(out, out_b) and torch.equal(lse, lse_b)
    wide = torch.full((2, 2, 140, 640), float("nan"), dtype=torch.bfloat16)
    wide[:, :, 4:132, 64:640] = x["q"]
    out_c, lse_c, _ = run(dict(x, q=wide.cuda()[:, :, 4:132, 64:640]))
    assert torch.equal(out, out_c) and torch.equal(lse, lse_c)


def test_captured_and_replayed():
    a = W.make_inputs_fp8(W.custom(6, 1, 128, 1, [700, 1, 64, 2000, 0, 130], causal=True), seed=1)
    b = W.make_inputs_fp8(W.custom(6, 1, 128, 1, [64, 1500, 0, 999, 300, 32], causal=True), seed=2, max_pages=a["max_pages"])
    pages = max(a["k8"].shape[0], b["k8"].shape[0])
    for x in (a, b):
        n = pages - x["k8"].shape[0]
        x["k8"] = torch.cat([x["k8"], torch.zeros(n, 64, 1, 576, dtype=torch.uint8)])
        x["k_scale"] = torch.cat([x["k_scale"], torch.ones(1, n, 64)], 1)
    names = ("q", "k8", "k_scale", "block_table", "cache_seqlens")
    d = {k: a[k].cuda() for k in names}
    parts = ops.num_parts_for(ops.device_sm_count(), 128, 1)
    ws = ops.new_workspace(ops.workspace_size(6, 1, 128, 1, parts), "cuda")

    def step():
        tile, splits = ops.get_mla_metadata(d["cache_seqlens"], 128, 1)
        return ops.mla_decode_paged_fp8_rows(d["q"], d["k8"], d["k_scale"], d["block_table"], d["cache_seqlens"], 512,
                                             tile, splits, causal=True, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for x in (b, a, b):
        for k in names:
            d[k].copy_(x[k])
        graph.replay()
        torch.cuda.synchronize()
        assert ops.query_status(ws) == ops.MLA_OK
        ref, ref_lse, _ = run(x)
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def test_two_graphs_side_by_side():
    # captured without a workspace: each graph has its own, so they may run at the same time
    xs = [W.make_inputs_fp8(W.custom(5, 1, 128, 1, [3000, 1, 500, 64, 900], causal=True), seed=s) for s in (1, 2)]
    runs = []
    for x in xs:
        ref, ref_lse, _ = run(x)
        d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
        tile, splits = ops.get_mla_metadata(d["cache_seqlens"], 128, 1)
        call = lambda: ops.mla_decode_paged_fp8_rows(d["q"], d["k8"], d["k_scale"], d["block_table"], d["cache_seqlens"],
                                                     512, tile, splits, softmax_scale=x["softmax_scale"], causal=True)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(8):
                got = call()
        runs.append((graph, got, ref, ref_lse, d, tile, splits, torch.cuda.Stream()))
    for _ in range(5):
        for graph, *_, stream in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, got, ref, ref_lse, *_ in runs:
        assert torch.equal(got[0], ref) and torch.equal(got[1], ref_lse)


def test_pages_outside_the_pool_leave_other_sequences_alone():
    x = W.make_inputs_fp8(W.custom(3, 1, 128, 1, [200, 300, 64], causal=True), seed=4)
    out, lse, _ = run(x)
    x["block_table"][1, 2], x["block_table"][1, 3] = 1 << 30, -7
    out2, lse2, _ = run(x)
    assert torch.equal(out2[[0, 2]], out[[0, 2]]) and torch.equal(lse2[[0, 2]], lse[[0, 2]])


@pytest.mark.parametrize("name", ["compute_bound", "causal_mtp", "skewed"])
def test_full_size_workloads(name):
    w = W.WORKLOADS[name]
    x = W.make_inputs_fp8(w, seed=0)
    worst, lse = parity(x)
    print(f"{name} over the FP8 cache: out {worst:.3f} of its tolerance, lse {lse:.2e}")


# --- keys whose scale is far above what they weigh -------------------------------------------------
#
# Tolerances relative to what each row holds itself.  The kernel's unit of v = P s follows the row's own
# largest P s: it lies in [2^6, 2^8] of them.  So v >= 2^-6, where its two terms keep it within 2^-8 (and
# its f16 form within 2^-11), for every key with p s >= 2^-12 of the row's largest; below, 2^-14 is at most
# 2^-20 of the largest (2^-11 in the code, for the largest of a part of the sequence).  A query element is
# exact when it is at least 2^-9 of its row's largest and within 2^-17 of the largest otherwise; each of
# the 36 accumulations of a score rounds by at most 2^-23 of sum|q k|.  A score off by d moves its
# probability by e^d, and all of them together.  2^-14 for the sums of PV (2^-23 for each of some 2^8
# accumulations and rescalings) and the exponentials.
def own_parity(x, num_parts=None):
    out, lse, _ = run(x, num_parts)
    q, h, g = x["q"].cuda().double(), x["h_kv"], x["h_q"] // x["h_kv"]
    k8, ks = x["k8"].cuda().view(torch.uint8), x["k_scale"].cuda().double()
    worst = 0.0
    for i, L in enumerate(x["cache_seqlens"].tolist()):
        pages = x["block_table"][i, :-(-L // 64)].long().cuda()
        for n in range(h):
            s = ks[n, pages].flatten()[:L]
            codes = k8[pages, :, n].view(torch.float8_e4m3fn).float().double().flatten(0, 1)[:L]
            c = codes * s[:, None]
            qn = q[i, :, n * g:(n + 1) * g]                                                   # [s_q, g, 576]
            top = qn.abs().amax(-1, keepdim=True)
            off = torch.where((qn.abs() >= 2.0 ** -9 * top) | (qn == 0), 0.0, 2.0 ** -17 * top)
            d = (off @ c.abs().t() + 36 * 2.0 ** -23 * (qn.abs() @ c.abs().t())) * x["softmax_scale"]
            rows = qn @ c.t() * x["softmax_scale"]
            if x["causal"]:
                keep = torch.arange(L, device="cuda") < L - (x["s_q"] - 1 - torch.arange(x["s_q"], device="cuda"))[:, None]
                rows = rows.masked_fill(~keep[:, None], -torch.inf)
            z = torch.logsumexp(rows, -1)
            p = torch.where(z[..., None] == -torch.inf, 0.0, (rows - z[..., None]).exp())
            ref = p @ c[:, :512]
            move = p * d.clamp_max(50).expm1()
            small = (p * s < 2.0 ** -11 * (p * s).amax(-1, keepdim=True)).double()
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -14) * (p @ c[:, :512].abs()) + \
                move @ c[:, :512].abs() + move.sum(-1, keepdim=True) * ref.abs() + \
                2.0 ** -20 * (p * s).amax(-1, keepdim=True) * (small @ codes[:, :512].abs()) + 1e-30
            err = ((out[i, :, n * g:(n + 1) * g].double() - ref).abs() / tol).max()
            worst = max(worst, float(err))
            gone = z == -torch.inf
            got = lse[i, n * g:(n + 1) * g].t().double()
            assert torch.equal(got == -torch.inf, gone)
            assert ((got - z).abs() <= 1e-4 * z.abs().clamp_min(1) + move.sum(-1))[~gone].all()
    assert worst <= 1, f"out off by {worst:.3f} of the tolerance"
    return worst


def key_at(x, b, t):
    return int(x["block_table"][b, t // 64]), t % 64


@pytest.mark.parametrize("std", [1.0, 1e-2, 1e-4])
@pytest.mark.parametrize("s_q,h_q", [(1, 17), (2, 64), (3, 64)])
@pytest.mark.parametrize("num_parts", [None, 1])
def test_rows_of_zeros_among_small_rows(std, s_q, h_q, num_parts):
    # the writer stores a row of zeros with scale 1, hundreds of thousands of times a small row's
    x = W.make_inputs(W.custom(3, s_q, h_q, 1, [1000, 130, 3], causal=True), seed=h_q + s_q)
    x["k_cache"][:x["num_pages"]] *= std
    x["q"] = (x["q"].float() / std).to(torch.bfloat16)
    for b, t in ((0, 5), (0, 700), (1, 129), (2, 0)):          # 129: only the last position sees it
        x["k_cache"][key_at(x, b, t)] = 0
    x["k8"], x["k_scale"] = W.to_fp8_cache(x["k_cache"])
    assert x["k_scale"][0][key_at(x, 1, 129)] == 1
    own_parity(x, num_parts)


@pytest.mark.parametrize("h_q", [17, 128])
@pytest.mark.parametrize("num_parts", [None, 1])
def test_large_keys_of_no_weight(h_q, num_parts):
    # scores of -20,000: no probability, but scales 5,000 times the other keys'
    x = W.make_inputs(W.custom(2, 1, h_q, 1, [600, 129], causal=False), seed=h_q)
    x["q"][..., 0] = 8
    for b, t in ((0, 17), (0, 40), (0, 300), (1, 0), (1, 128)):
        row = x["k_cache"][key_at(x, b, t)]
        row *= 2.0 ** 10
        row[..., 0] = -2.0 ** 16
    x["k8"], x["k_scale"] = W.to_fp8_cache(x["k_cache"])
    own_parity(x, num_parts)


@pytest.mark.parametrize("h_q,s_q", [(17, 1), (128, 1), (64, 3)])
@pytest.mark.parametrize("num_parts", [None, 1])
@pytest.mark.parametrize("span", [4, 8])
def test_scales_against_probabilities(h_q, s_q, num_parts, span):
    # scales 2^e with e up to +-span, and scores that fall with e: p s is spread by 2^(span / 2) both ways
    # around one, led by large keys in some places and by small ones in others
    x = W.make_inputs_fp8(W.custom(3, s_q, h_q, 1, [900, 190, 64], causal=True), seed=span + h_q)
    g = torch.Generator().manual_seed(span)
    n = x["k8"].shape[0]
    e = torch.randint(-span, span + 1, (n, 64), generator=g).float()
    e[: n // 2] = e[: n // 2].sort(-1).values                  # growing within a page, and any order
    x["k_scale"] = torch.exp2(e)[None].contiguous()
    score = -math.log(2.0) * e * (0.5 + torch.rand(n, 64, generator=g))
    # only column 512 of the query is not zero: the score is q_512 * code_512 * scale / 24, and 2^(span - 1)
    # in it reaches the scores of the smallest scales with codes below 448
    x["softmax_scale"] = 1 / 24
    x["q"].zero_()
    x["q"][..., 512] = (0.75 + 0.5 * torch.rand(x["q"].shape[:3], generator=g)) * 2.0 ** (span - 1)
    code = (24 * 2.0 ** (1 - span) * score / torch.exp2(e)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    x["k8"][:, :, 0, 512] = code
    own_parity(x, num_parts)


def test_small_query_elements():
    """One key of ones, so the LSE is the score, sum(q) / 24, beside one query element of 1.0 that meets a
    zero.  1.0 becomes 128: an element of 2^-9 or more is 2^-2 or more there and exact; 2^-10 (1 + 2^-7) is
    2^-3 + 2^-10, half a step of 2^-9 off, 2^-17 of the largest, and the next even code is 2^-3.
    The score's 36 accumulations round by 2^-23 of it each; 2e-6 for the LSE's log2, sum and product."""
    x = W.make_inputs_fp8(W.custom(1, 1, 128, 1, [1], causal=False), seed=1)
    x["k8"].fill_(0x38)
    x["k8"][..., 0] = 0
    x["k_scale"].fill_(1.0)
    x["softmax_scale"] = 1 / 24
    g = torch.Generator().manual_seed(2)
    x["q"][0, 0, :64] = 2.0 ** -9 * (1 + torch.randint(0, 128, (64, 576), generator=g) / 128)
    x["q"][0, 0, 64:] = 2.0 ** -10 * (1 + 2.0 ** -7)
    x["q"][..., 0] = 1.0
    want = x["q"][0, 0, :, 1:].double().sum(-1).cuda() / 24
    _, lse, _ = run(x)
    off = (lse[0, :, 0].double() - want).abs()
    slack = 36 * 2.0 ** -23 * want + 2e-6
    assert (off[:64] <= slack[:64]).all()
    assert (off[64:] <= 2.0 ** -17 * 575 / 24 + slack[64:]).all()
    assert (off[64:] > 2.0 ** -18 * 575 / 24 + slack[64:]).all()         # not within half of that


@pytest.mark.parametrize("num_parts", [None, 1, 3])
def test_a_key_of_nan_stays_in_its_sequence(num_parts):
    x = W.make_inputs_fp8(W.custom(4, 2, 64, 1, [300, 1000, 70, 129], causal=True), seed=6)
    out, lse, _ = run(x, num_parts)
    x["k8"] = x["k8"].clone()
    x["k8"][key_at(x, 1, 999)] = 0x7f                          # only the last position sees it
    out2, lse2, _ = run(x, num_parts)
    keep = [0, 2, 3]
    assert torch.equal(out2[keep], out[keep]) and torch.equal(lse2[keep], lse[keep])
    assert torch.isnan(out2[1, 1]).all() and torch.isnan(lse2[1, :, 1]).all()
