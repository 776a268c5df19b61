"""Writing the latent cache (mla_cache_slots, mla_cache_write, mla_cache_write_fp8) and reading
it back (mla_cache_read, mla_cache_read_fp8) against the same written out in fp64.

Tolerances.  The norm's factor in fp32: a sum of 512 squares as 16 terms per lane and five
pairwise steps, relative error <= 21 * 2^-24, halved by the square root, plus rsqrtf's 2^-22.5
and the products': 1.5e-6 of the value.  The rotation: 5e-7 * (|x0| + |x1|) (test_rope_gpu).
Rounding: bf16 half a step, 2^-8 of the value; E4M3 2^-4 of the value, or half its smallest
step, 2^-10, times the scale, widened by 2^-18 for quotients next to the middle of two codes."""

import numpy as np
import pytest
import torch

from paged_mla_decode_11_b200 import ops
from paged_mla_decode_11_b200 import workloads as W

pytestmark = pytest.mark.gpu


def draw(T, h_kv, dtype, pages, seed=0, norm=True, rope=True, spread=False, pos_type=torch.int32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    both = torch.randn(T, h_kv, 576, generator=g, device="cuda")
    if spread:  # rows of very different sizes
        both = both * torch.exp2(torch.randint(-12, 12, (T, h_kv, 1), generator=g, device="cuda").float())
    both = both.to(dtype)
    slots = torch.randperm(pages * 64, generator=g, device="cuda")[:T]
    kw = {}
    if norm:
        kw.update(norm_weight=(1 + 0.2 * torch.randn(512, generator=g, device="cuda")).to(dtype), eps=1e-5)
    if rope:
        kw.update(positions=torch.randint(0, 1 << 20, (T,), generator=g, device="cuda").to(pos_type),
                  inv_freq=ops.rope_frequencies(64, scaling="yarn", factor=40.0, device="cuda"), magnitude=1.1)
    return both, slots, kw


def formed(both, kw, interleaved=True):
    """The rows in fp64 and the error their fp32 forms may have."""
    y = both.double().clone()
    tol = torch.zeros_like(y)
    if "norm_weight" in kw:
        x = y[..., :512]
        y[..., :512] = x * kw["norm_weight"].double() / (x.square().mean(-1, keepdim=True) + kw["eps"]).sqrt()
        tol[..., :512] = 1.5e-6 * y[..., :512].abs()
    if "positions" in kw:
        a = kw["positions"].double()[:, None, None] * kw["inv_freq"]
        at = (slice(512, 576, 2), slice(513, 576, 2)) if interleaved else (slice(512, 544), slice(544, 576))
        x0, x1 = both[..., at[0]].double(), both[..., at[1]].double()
        y[..., at[0]] = kw["magnitude"] * (x0 * a.cos() - x1 * a.sin())
        y[..., at[1]] = kw["magnitude"] * (x0 * a.sin() + x1 * a.cos())
        for s in at:
            tol[..., s] = 5e-7 * kw["magnitude"] * (x0.abs() + x1.abs())
    return y, tol


def check_bf16(got, both, kw, interleaved=True):
    y, tol = formed(both, kw, interleaved)
    assert ((got.double() - y).abs() <= tol + 2.0 ** -8 * (y.abs() + tol)).all()


def check_fp8(codes, scale, both, kw, interleaved=True):
    y, tol = formed(both, kw, interleaved)
    amax, at = y.abs().max(-1)
    want = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    off = tol.amax(-1) / 448 + 2.0 ** -22 * want
    assert ((scale.double() - want).abs() <= off).all()
    v = codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None]
    half = torch.maximum(2.0 ** -4 * (y.abs() + tol), 2.0 ** -10 * scale.double()[..., None])
    assert ((v - y).abs() <= tol + half * (1 + 2.0 ** -18)).all()
    assert (codes.view(torch.float8_e4m3fn).float().abs().amax(-1)[amax > 0] == 448).all()


@pytest.mark.parametrize("T,h_kv", [(1, 1), (7, 1), (64, 1), (65, 2), (1300, 1), (33, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("norm,rope,interleaved", [(True, True, True), (True, True, False), (False, True, True),
                                                   (True, False, True), (False, False, True)])
def test_write_then_read(T, h_kv, dtype, norm, rope, interleaved):
    pages = T // 64 + 3
    both, slots, kw = draw(T, h_kv, dtype, pages, seed=T, norm=norm, rope=rope,
                           pos_type=torch.int64 if T % 2 else torch.int32)
    how = dict(kw, interleaved=interleaved)
    g = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.randn(pages, 64, h_kv, 576, generator=g, device="cuda").to(torch.bfloat16)
    k8 = torch.randint(0, 120, pool.shape, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    ks = torch.rand(h_kv, pages, 64, generator=g, device="cuda")
    pool0, k80, ks0 = pool.clone(), k8.clone(), ks.clone()
    ops.mla_cache_write(both[..., :512], both[..., 512:], slots, pool, **how)
    ops.mla_cache_write_fp8(both[..., :512], both[..., 512:], slots, k8, ks, **how)
    rows, codes = pool.view(-1, h_kv, 576), k8.view(-1, h_kv, 576)
    scale = ks.view(h_kv, -1).t()
    check_bf16(rows[slots], both, kw, interleaved)
    check_fp8(codes[slots], scale[slots], both, kw, interleaved)
    # every other row as it was
    other = torch.ones(pages * 64, dtype=torch.bool, device="cuda")
    other[slots] = False
    assert torch.equal(rows[other], pool0.view(-1, h_kv, 576)[other])
    assert torch.equal(codes[other], k80.view(-1, h_kv, 576)[other])
    assert torch.equal(scale[other], ks0.view(h_kv, -1).t()[other])
    # and read back: bf16 rows as they are, FP8 rows as the rounded product
    assert torch.equal(ops.mla_cache_read(pool, slots), rows[slots])
    back = ops.mla_cache_read_fp8(k8, ks, slots)
    want = codes[slots].view(torch.float8_e4m3fn).double() * scale[slots].double()[..., None]
    assert ((back.double() - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -15) * want.abs()).all()


def test_row_sizes_and_zero_rows():
    both, slots, kw = draw(300, 1, torch.float32, 6, seed=5, norm=False, spread=True)
    both[3] = 0
    both[4, :, 1:] = 0
    both[4, :, 0] = 1e-44                                   # a subnormal row: the scale underflows
    both[5] *= 1e-36 / both[5].abs().max()
    both[6] *= 3e38 / both[6].abs().max()
    kw = dict(kw, magnitude=1.0)
    k8 = torch.full((6, 64, 1, 576), 0x7f, dtype=torch.uint8, device="cuda")
    ks = torch.full((1, 6, 64), float("nan"), device="cuda")
    ops.mla_cache_write_fp8(both[..., :512], both[..., 512:], slots, k8, ks, **kw)
    codes, scale = k8.view(-1, 1, 576)[slots], ks.view(1, -1).t()[slots]
    assert scale[3] == 1 and (codes[3] & 0x7f == 0).all()
    assert scale[4] == 1 and (codes[4] & 0x7f == 0).all()
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[3:5] = False
    check_fp8(codes[keep], scale[keep], both[keep], dict(kw, positions=kw["positions"][keep]))


def test_non_finite_values_become_nan_codes_and_leave_the_scale():
    both, slots, _ = draw(4, 1, torch.float32, 1, seed=6, norm=False, rope=False)
    clean = both.clone()
    both[1, 0, 17], both[2, 0, 570], both[3] = float("nan"), float("-inf"), float("inf")
    clean[1, 0, 17], clean[2, 0, 570] = 0, 0
    k8 = torch.zeros(1, 64, 1, 576, dtype=torch.float8_e4m3fn, device="cuda")
    ks = torch.zeros(1, 1, 64, device="cuda")
    ops.mla_cache_write_fp8(both[..., :512], both[..., 512:], slots, k8, ks)
    codes, scale = k8.view(torch.uint8).view(-1, 1, 576)[slots], ks.view(1, -1).t()[slots]
    bad = ~torch.isfinite(both)
    assert ((codes & 0x7f == 0x7f) == bad).all() and scale[3] == 1
    fixed = torch.where(bad, torch.zeros_like(codes), codes)
    check_fp8(fixed[:3], scale[:3], clean[:3], {})


@pytest.mark.parametrize("fp8", [False, True])
def test_slots_outside_the_pool(fp8):
    both, slots, kw = draw(40, 2, torch.bfloat16, 2, seed=7)
    slots[3], slots[9], slots[10], slots[39] = -1, 128, 2 ** 40, -2 ** 62
    pool = torch.zeros(2, 64, 2, 576, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    ks = torch.zeros(2, 2, 64, device="cuda")
    args = (pool, ks) if fp8 else (pool,)
    (ops.mla_cache_write_fp8 if fp8 else ops.mla_cache_write)(both[..., :512], both[..., 512:], slots, *args, **kw)
    fine = (slots >= 0) & (slots < 128)
    assert int(fine.sum()) == 36
    assert int((pool.view(128, -1) != 0).any(-1).sum()) == 36
    back = (ops.mla_cache_read_fp8 if fp8 else ops.mla_cache_read)(*args, slots)
    assert (back[~fine] == 0).all() and (back[fine] != 0).any(-1).all()
    # a slot may be read more than once, into rows of a wider buffer that is left alone elsewhere
    wide = torch.full((6, 3, 600), 7.0, dtype=torch.bfloat16, device="cuda")
    twice = slots[fine][:3].repeat(2)
    (ops.mla_cache_read_fp8 if fp8 else ops.mla_cache_read)(*args, twice, out=wide[:, :2, 8:584])
    assert torch.equal(wide[:3, :2, 8:584], wide[3:, :2, 8:584]) and torch.equal(wide[:3, :2, 8:584], back[fine][:3])
    assert (wide[:, 2] == 7).all() and (wide[..., :8] == 7).all() and (wide[..., 584:] == 7).all()


def test_slots_follow_the_block_table():
    lens, new = [70, 0, 64, 5, 200, 3], [6, 0, 64, 5, 0, 5]
    table = torch.randperm(40)[:24].to(torch.int32).view(6, 4)
    table[4, 3] = 99
    ptr = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    T = int(ptr[-1]) + 9                                    # nine padding tokens
    slots, pos = ops.mla_cache_slots(table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), ptr.cuda(), 40, T)
    want_s, want_p = [], []
    for b, (L, n) in enumerate(zip(lens, new)):
        for i in range(n):
            x = L - n + i
            ok = x >= 0                                     # sequence 5 has fewer entries than new tokens
            want_s.append(int(table[b, x // 64]) * 64 + x % 64 if ok else -1)
            want_p.append(x if ok else 0)
    assert slots.tolist() == want_s + [-1] * 9 and pos.tolist() == want_p + [0] * 9
    # pages outside the pool and positions past the table's width
    ptr = torch.tensor([0, 200, 230], dtype=torch.int32).cuda()
    slots, pos = ops.mla_cache_slots(table[[4, 0], :].cuda()[:, :4], torch.tensor([200, 270], dtype=torch.int32).cuda(),
                                     ptr, 40, 230)
    x = torch.arange(200)
    want = torch.where(x < 192, table[4].long()[x // 64] * 64 + x % 64, -1)
    assert torch.equal(slots[:200].cpu(), want)
    x = torch.arange(240, 270)
    want = torch.where(x < 256, table[0].long()[(x // 64).clamp_max(3)] * 64 + x % 64, -1)
    assert torch.equal(slots[200:].cpu(), want)


@pytest.mark.parametrize("b", [1, 2, 700])
def test_slots_many_sequences(b):
    g = torch.Generator().manual_seed(b)
    new = torch.randint(0, 4, (b,), generator=g)
    lens = new + torch.randint(0, 500, (b,), generator=g)
    table = torch.randperm(b * 8, generator=g).to(torch.int32).view(b, 8)
    ptr = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).to(torch.int32)
    T = int(ptr[-1])
    slots, pos = ops.mla_cache_slots(table.cuda(), lens.to(torch.int32).cuda(), ptr.cuda(), b * 8, T)
    seq = torch.repeat_interleave(torch.arange(b), new)
    x = lens[seq] - new[seq] + torch.arange(T) - ptr[:-1].long()[seq]
    assert torch.equal(pos.cpu().long(), x)
    assert torch.equal(slots.cpu(), table[seq, x // 64].long() * 64 + x % 64)


def test_empty_calls_and_a_long_pool():
    kc = torch.zeros(1, 64, 1, 576, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    ops.mla_cache_write(torch.empty(0, 1, 512, dtype=torch.bfloat16, device="cuda"),
                        torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda"), none, kc)
    assert ops.mla_cache_read(kc, none).shape == (0, 1, 576)
    # byte offsets above 2^32: a pool of 5.2 GB
    pages = 71000
    pool = torch.zeros(pages, 64, 1, 576, dtype=torch.bfloat16, device="cuda")
    both, _, kw = draw(3, 1, torch.bfloat16, 1, seed=2)
    slots = torch.tensor([pages * 64 - 1, 0, 3_800_000], device="cuda")
    ops.mla_cache_write(both[..., :512], both[..., 512:], slots, pool, **kw)
    check_bf16(pool.view(-1, 1, 576)[slots], both, kw)
    assert torch.equal(ops.mla_cache_read(pool, slots), pool.view(-1, 1, 576)[slots])
    assert int((pool.view(-1, 576)[:, 0] != 0).sum()) == 3


def test_written_cache_decodes_like_the_generators():
    """slots -> write (FP8) -> decode, captured into one graph and replayed on new inputs: the
    written cache equals the input generator's FP8 format, so the decode agrees bit for bit."""
    x = W.make_inputs(W.custom(3, 1, 16, 1, [130, 1, 64], causal=True), seed=3)
    k8, ks = W.to_fp8_cache(x["k_cache"])
    pages = k8.shape[0]
    table, lens = x["block_table"].cuda(), x["cache_seqlens"].cuda()
    ptr = torch.tensor([0, 130, 131, 195], dtype=torch.int32, device="cuda")
    src = torch.zeros(200, 1, 576, dtype=torch.bfloat16, device="cuda")
    mine, scale = torch.zeros(pages, 64, 1, 576, dtype=torch.uint8, device="cuda"), torch.ones(1, pages, 64, device="cuda")
    q = x["q"].cuda()
    ws = ops.new_workspace(1 << 24, "cuda")
    plan, splits = ops.get_mla_metadata(lens, 16, 1)
    out, lse = torch.empty(3, 1, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 16, 1, device="cuda")

    def step():
        slots, _ = ops.mla_cache_slots(table, lens, ptr, pages, 200)
        ops.mla_cache_write_fp8(src[..., :512], src[..., 512:], slots, mine, scale)
        ops.mla_decode_paged_fp8(q, mine, scale, table, lens, 512, plan, splits, causal=True, workspace=ws, out=out, lse=lse)

    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    slots, _ = ops.mla_cache_slots(table, lens, ptr, pages, 195)
    src[:195] = x["k_cache"].cuda().view(-1, 1, 576)[slots]
    graph.replay()
    torch.cuda.synchronize()
    assert ops.query_status(ws) == ops.MLA_OK
    assert torch.equal(scale.view(-1)[slots].cpu(), ks.view(-1)[slots.cpu()])
    a = mine.view(-1, 576)[slots].view(torch.float8_e4m3fn).float().cpu()
    b = k8.view(-1, 576)[slots.cpu()].view(torch.float8_e4m3fn).float()
    assert (a != b).float().mean() <= 1e-4          # quotients next to the middle of two codes
    ref, ref_lse = ops.mla_decode_paged_fp8(q, mine, scale, table, lens, 512, plan, splits, causal=True)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_of_single_elements_do_not_matter(dtype):
    # one token of one latent head, cut from rows of an odd width: neither stride is ever stepped over
    both, slots, kw = draw(1, 1, dtype, 3, seed=8)
    odd = torch.zeros(1, 7, 577, dtype=dtype, device="cuda")
    odd[:, :1, :576] = both
    row = odd[:, :1, :576]
    assert row.stride() == (7 * 577, 577, 1)
    pools = [torch.zeros(3, 64, 1, 576, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for pool, r in zip(pools, (both, row)):
        ops.mla_cache_write(r[..., :512], r[..., 512:], slots, pool, **kw)
    assert torch.equal(*pools) and pools[0].any()
    caches = [(torch.zeros(3, 64, 1, 576, dtype=torch.uint8, device="cuda"), torch.ones(1, 3, 64, device="cuda")) for _ in range(2)]
    for (k8, ks), r in zip(caches, (both, row)):
        ops.mla_cache_write_fp8(r[..., :512], r[..., 512:], slots, k8, ks, **kw)
    assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
    out = torch.zeros(1, 7, 577, dtype=torch.bfloat16, device="cuda")
    ops.mla_cache_read(pools[0], slots, out=out[:, :1, :576])
    assert torch.equal(out[:, :1, :576], ops.mla_cache_read(pools[0], slots)) and not out[:, 1:].any()
    x = odd[:, :1, 512:576]
    assert torch.equal(ops.mla_rope(x, kw["positions"], kw["inv_freq"]),
                       ops.mla_rope(x.contiguous(), kw["positions"], kw["inv_freq"]))
    place = odd[:, :1, 512:576]
    want = ops.mla_rope(place, kw["positions"], kw["inv_freq"])
    ops.mla_rope(place, kw["positions"], kw["inv_freq"], out=place)
    assert torch.equal(place, want) and not odd[:, 1:].any() and not odd[..., 576].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("exponent", [-30, 0, 14])
def test_rows_as_given_are_correctly_rounded_quotients(dtype, exponent):
    """Without a norm the codes are exactly those of the IEEE quotient row / scale: the corrected
    product is the correctly rounded quotient (and below 1e-24 the kernel divides)."""
    g = torch.Generator(device="cuda").manual_seed(exponent + 40)
    T = 20000
    both = torch.randn(T, 1, 576, generator=g, device="cuda")
    if dtype == torch.float32:
        both *= torch.exp2(torch.randint(-60, 61, (T, 1, 1), generator=g, device="cuda").float())
    both = (both * 2.0 ** (exponent / 2 if dtype == torch.float16 else exponent)).to(dtype)
    slots = torch.randperm(320 * 64, generator=g, device="cuda")[:T]
    k8 = torch.zeros(320, 64, 1, 576, dtype=torch.uint8, device="cuda")
    ks = torch.ones(1, 320, 64, device="cuda")
    ops.mla_cache_write_fp8(both[..., :512], both[..., 512:], slots, k8, ks)
    rows = both.float()
    amax = rows.abs().amax(-1)
    # numpy divides; torch on CUDA multiplies by the rounded 1 / 448 of a Python scalar
    scale = torch.from_numpy(amax.cpu().numpy() / np.float32(448)).cuda()
    scale[scale == 0] = 1
    assert torch.equal(ks.view(1, -1).t()[slots], scale)
    want = (rows / scale[..., None]).to(torch.float8_e4m3fn).float()
    # as values: the corrected product of -0 is (-0 - 0) y + -0, a zero of the other sign
    assert torch.equal(k8.view(-1, 1, 576)[slots].view(torch.float8_e4m3fn).float(), want)
