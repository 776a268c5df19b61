"""Host-side checks, without a GPU, of the operators around the decode: what the marshalling
module and the C ABI refuse before anything reaches a device, and the frequency formulas."""

import ctypes
import math

import pytest
import torch

from paged_mla_decode_11_b200 import build as B
from paged_mla_decode_11_b200 import ops

bf, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    ops.load_binding()


def z(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


def rope_args(**over):
    a = dict(x=z(5, 4, 64), positions=z(5, dtype=i64), inv_freq=ops.rope_frequencies(64))
    a.update(over)
    return a


@pytest.mark.parametrize("over,exc,msg", [
    (dict(x=[1.0]), TypeError, "x must be a tensor"),
    (dict(x=z(5, 4, 64, dtype=torch.float64)), TypeError, "x must be bf16"),
    (dict(x=z(5, 64)), ValueError, "tokens, heads, width"),
    (dict(x=z(5, 4, 128)[..., ::2]), ValueError, "last dimension"),
    (dict(x=z(5, 4, 63)), ValueError, "inv_freq"),
    (dict(inv_freq=ops.rope_frequencies(64).float()), TypeError, "inv_freq must be"),
    (dict(inv_freq=torch.zeros(0, dtype=torch.float64)), ValueError, "inv_freq"),
    (dict(inv_freq=torch.zeros(64, dtype=torch.float64)[::2]), ValueError, "inv_freq"),
    (dict(positions=z(4, dtype=i64)), ValueError, "positions"),
    (dict(positions=z(5, dtype=f32)), TypeError, "positions must be int32 or int64"),
    (dict(positions=z(10, dtype=i64)[::2]), ValueError, "positions"),
    (dict(out=z(5, 4, 32)), ValueError, "x's shape"),
    (dict(out=z(5, 4, 64, dtype=f32)), TypeError, "out must be"),
    (dict(out=z(1, 4, 64).expand(5, 4, 64)), ValueError, "rows of out"),
    (dict(magnitude="m"), TypeError, "number"),
    (dict(), ValueError, "CUDA tensor"),                       # all else is in order
])
def test_rope_refusals(over, exc, msg):
    with pytest.raises(exc, match=msg):
        ops.mla_rope(**rope_args(**over))


def test_rope_with_a_gradient_refuses_an_output_and_checks_alike():
    x = z(5, 4, 64).requires_grad_()
    with pytest.raises(ValueError, match="needs a gradient"):
        ops.mla_rope(**rope_args(x=x, out=z(5, 4, 64)))
    with pytest.raises(ValueError, match="positions"):
        ops.mla_rope(**rope_args(x=x, positions=z(4, dtype=i64)))
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.mla_rope(**rope_args(x=x))
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensor"):   # passes the checks
        ops.mla_rope(**rope_args(x=x, out=z(5, 4, 64)))


def test_rope_refuses_partly_overlapping_rows():
    base = z(5, 4, 200)
    with pytest.raises(ValueError, match="must not overlap it"):
        ops.mla_rope(**rope_args(x=base[..., :64], out=base[..., 8:72]))
    with pytest.raises(ValueError, match="CUDA tensor"):       # in place passes the checks
        x = base[..., 64:128]
        ops.mla_rope(**rope_args(x=x, out=x))
    with pytest.raises(ValueError, match="rows of out"):       # heads closer than their width
        ops.mla_rope(**rope_args(out=torch.as_strided(z(5000), (5, 4, 64), (256, 32, 1))))
    with pytest.raises(ValueError, match="CUDA tensor"):       # head-major rows are apart
        ops.mla_rope(**rope_args(out=z(4, 5, 64).transpose(0, 1)))


def write_args(fp8=False, **over):
    both = z(6, 1, 576)
    a = dict(latent=both[..., :512], rope=both[..., 512:], slots=z(6, dtype=i64))
    a.update(dict(k8=z(3, 64, 1, 576, dtype=torch.uint8), k_scale=z(1, 3, 64, dtype=f32)) if fp8 else
             dict(k_cache=z(3, 64, 1, 576)))
    a.update(over)
    return a


@pytest.mark.parametrize("over,exc,msg", [
    (dict(latent=z(6, 1, 512, dtype=torch.int8)), TypeError, "latent must be"),
    (dict(rope=z(6, 1, 64, dtype=f32)), TypeError, "rope must be"),
    (dict(latent=z(6, 512)), ValueError, "latent must be"),
    (dict(latent=z(6, 1, 576)), ValueError, "latent must be"),
    (dict(rope=z(6, 1, 32)), ValueError, "rope must be"),
    (dict(rope=z(5, 1, 64)), ValueError, "rope must be"),
    (dict(latent=z(6, 1, 1024)[..., ::2]), ValueError, "last dimensions"),
    (dict(slots=z(6, dtype=i32)), TypeError, "slots must be"),
    (dict(slots=z(7, dtype=i64)), ValueError, "slots must be"),
    (dict(norm_weight=z(512, dtype=f32)), TypeError, "norm_weight"),
    (dict(norm_weight=z(576)), ValueError, "norm_weight"),
    (dict(positions=z(6, dtype=i32)), ValueError, "positions need inv_freq"),
    (dict(inv_freq=ops.rope_frequencies(64)), ValueError, "inv_freq needs positions"),
    (dict(positions=z(6, dtype=i32), inv_freq=ops.rope_frequencies(32)), ValueError, "inv_freq"),
    (dict(positions=z(5, dtype=i32), inv_freq=ops.rope_frequencies(64)), ValueError, "positions"),
    (dict(), ValueError, "CUDA tensor"),
])
@pytest.mark.parametrize("fp8", [False, True])
def test_write_refusals(over, exc, msg, fp8):
    with pytest.raises(exc, match=msg):
        (ops.mla_cache_write_fp8 if fp8 else ops.mla_cache_write)(**write_args(fp8, **over))


@pytest.mark.parametrize("call,over,exc,msg", [
    ("write", dict(k_cache=z(3, 64, 1, 576, dtype=f32)), TypeError, "k_cache must be bf16"),
    ("write", dict(k_cache=z(3, 64, 2, 576)), ValueError, "h_kv"),
    ("write", dict(k_cache=z(3, 32, 1, 576)), ValueError, "the cache must be"),
    ("write", dict(k_cache=z(3, 64, 1, 600)[..., :576]), ValueError, "the cache must be"),
    ("write8", dict(k8=z(3, 64, 1, 576)), TypeError, "k8 must be"),
    ("write8", dict(k_scale=z(3, 64, 1, dtype=f32)), ValueError, "k_scale"),
    ("write8", dict(k_scale=z(1, 3, 64)), TypeError, "k_scale"),
    ("read", dict(k_cache=z(3, 64, 1, 576, dtype=torch.uint8)), TypeError, "k_cache must be bf16"),
    ("read", dict(slots=z(2, 2, dtype=i64)), ValueError, "slots must be"),
    ("read", dict(slots=z(2, dtype=i32)), TypeError, "slots must be"),
    ("read", dict(out=z(6, 1, 512)), ValueError, "out must be"),
    ("read", dict(out=z(6, 1, 576, dtype=f32)), TypeError, "out must be"),
    ("read", dict(out=z(1, 1, 576).expand(6, 1, 576)), ValueError, "rows of out"),
    ("read", dict(), ValueError, "CUDA tensor"),
    ("read8", dict(k_scale=z(2, 3, 64, dtype=f32)), ValueError, "k_scale"),
    ("read8", dict(), ValueError, "CUDA tensor"),
])
def test_pool_refusals(call, over, exc, msg):
    a = write_args(call.endswith("8"), **over)
    if call.startswith("read"):
        a = {k: v for k, v in a.items() if k not in ("latent", "rope")}
    fn = dict(write=ops.mla_cache_write, write8=ops.mla_cache_write_fp8, read=ops.mla_cache_read, read8=ops.mla_cache_read_fp8)[call]
    with pytest.raises(exc, match=msg):
        fn(**a)


def test_write_refuses_rows_of_the_cache_itself():
    pool = z(3, 64, 1, 576)
    rows = pool.view(192, 1, 576)[10:16]
    for over in (dict(latent=rows[..., :512]), dict(rope=rows[..., 512:])):
        with pytest.raises(ValueError, match="must not overlap the cache"):
            ops.mla_cache_write(**write_args(k_cache=pool, **over))
    with pytest.raises(ValueError, match="CUDA tensor"):       # other rows of the same storage
        both = z(4, 64, 1, 576)
        ops.mla_cache_write(**write_args(k_cache=both[:3], latent=both[3, :6, :, :512], rope=both[3, :6, :, 512:]))


def test_read_refuses_an_output_inside_the_cache():
    pool = z(3, 64, 1, 576)
    with pytest.raises(ValueError, match="overlap the cache"):
        ops.mla_cache_read(pool, z(6, dtype=i64), out=pool.view(-1, 1, 576)[10:16])


@pytest.mark.parametrize("over,exc,msg", [
    (dict(block_table=z(3, 4, dtype=i64)), TypeError, "block_table"),
    (dict(block_table=z(4, 3, dtype=i32).t()), ValueError, "block_table"),
    (dict(cache_seqlens=z(2, dtype=i32)), ValueError, "cache_seqlens"),
    (dict(row_ptr=z(3, dtype=i32)), ValueError, "row_ptr"),
    (dict(tokens=-1), ValueError, "tokens"),
    (dict(slots=z(9, dtype=i64)), ValueError, "slots"),
    (dict(positions=z(10, dtype=i64)), TypeError, "positions"),
    (dict(), ValueError, "CUDA tensor"),
])
def test_slot_refusals(over, exc, msg):
    a = dict(block_table=z(3, 4, dtype=i32), cache_seqlens=z(3, dtype=i32), row_ptr=z(4, dtype=i32), num_pages=12, tokens=10)
    a.update(over)
    with pytest.raises(exc, match=msg):
        ops.mla_cache_slots(**a)


@pytest.mark.parametrize("over,exc,msg", [
    (dict(target_probs=z(2, 4, 9, dtype=torch.int32)), TypeError, "target_probs"),
    (dict(target_probs=z(2, 1, 9, dtype=f32)), ValueError, "at least one draft"),
    (dict(target_probs=z(2, 4, 18, dtype=f32)[..., ::2]), ValueError, "last dimension"),
    (dict(draft_tokens=z(2, 3, dtype=i64)), TypeError, "draft_tokens"),
    (dict(draft_tokens=z(2, 4, dtype=i32)), ValueError, "draft_tokens"),
    (dict(uniform=z(3, 2, dtype=f32).t()), ValueError, "uniform"),
    (dict(uniform_new=z(3, dtype=f32)), ValueError, "uniform_new"),
    (dict(draft_probs=z(2, 3, 9)), TypeError, "draft_probs"),
    (dict(draft_probs=z(2, 4, 9, dtype=f32)), ValueError, "draft_probs"),
    (dict(num_drafts=z(2, dtype=i64)), TypeError, "num_drafts"),
    (dict(num_drafts=z(1, dtype=i32)), ValueError, "num_drafts"),
    (dict(), ValueError, "CUDA tensor"),
])
def test_verify_refusals(over, exc, msg):
    a = dict(target_probs=z(2, 4, 9, dtype=f32), draft_tokens=z(2, 3, dtype=i32), uniform=z(2, 3, dtype=f32),
             uniform_new=z(2, dtype=f32))
    a.update(over)
    with pytest.raises(exc, match=msg):
        ops.mla_verify_draft(**a)


@pytest.mark.parametrize("over,exc,msg", [
    (dict(q=z(3, 1, 128, 576, dtype=f32)), TypeError, "q must be"),
    (dict(q=z(3, 128, 576)), ValueError, "4-D"),
    (dict(q=z(3, 1, 128, 512)), ValueError, "latent width"),
    (dict(q=z(3, 1, 128, 1152)[..., ::2]), ValueError, "last dimension"),
    (dict(k8=z(10, 64, 1, 576)), TypeError, "k8 must be"),
    (dict(k8=z(10, 64, 1, 600, dtype=torch.uint8)[..., :576]), ValueError, "the cache must be"),
    (dict(k_scale=z(1, 9, 64, dtype=f32)), ValueError, "k_scale"),
    (dict(block_table=z(2, 6, dtype=i32)), ValueError, "block_table"),
    (dict(block_table=z(6, 3, dtype=i32).t()), ValueError, "block_table"),
    (dict(cache_seqlens=z(4, dtype=i32)), ValueError, "cache_seqlens"),
    (dict(tile_metadata=z(5, 7, dtype=i32)), ValueError, "tile_metadata"),
    (dict(num_splits=z(3, dtype=i32)), ValueError, "num_splits"),
    (dict(num_splits=z(4, dtype=i64)), TypeError, "num_splits"),
    (dict(out=z(3, 1, 128, 256)), ValueError, "out must be"),
    (dict(lse=z(3, 1, 128, dtype=f32)), ValueError, "lse must be"),
    (dict(dv=-1), ValueError, "out of range"),
    (dict(softmax_scale="s"), TypeError, "number"),
    (dict(), ValueError, "CUDA tensor"),
])
def test_decode_rows_refusals(over, exc, msg):
    a = dict(q=z(3, 1, 128, 576), k8=z(10, 64, 1, 576, dtype=torch.uint8), k_scale=z(1, 10, 64, dtype=f32),
             block_table=z(3, 6, dtype=i32), cache_seqlens=z(3, dtype=i32), dv=512, tile_metadata=z(5, 8, dtype=i32),
             num_splits=z(4, dtype=i32))
    a.update(over)
    with pytest.raises(exc, match=msg):
        ops.mla_decode_paged_fp8_rows(**a)


def test_c_abi_refusals():
    """Every refusal below comes before any device call; the addresses are never read."""
    lib = ops.load_library()
    s2 = (ctypes.c_int64 * 2)(576, 576)
    odd = (ctypes.c_int64 * 2)(577, 576)
    neg = (ctypes.c_int64 * 2)(-576, 576)
    err = lib.mla_last_error_string

    def rope(x=16, xs=s2, dtype=0, T=4, H=2, D=64, n=32, pos=16, f=16, m=1.0, flags=0, out=32, os=s2):
        return lib.mla_rope(x, xs, dtype, T, H, D, n, pos, f, m, flags, out, os, None)
    assert rope(dtype=3) == -1 and b"element type" in err()
    assert rope(n=0) == -1 and rope(n=33) == -1 and rope(D=70000, n=2) == -1
    assert rope(flags=8) == -1 and b"flags" in err()
    assert rope(m=math.inf) == -1 and b"magnitude" in err()
    assert rope(x=None) == -1 and rope(pos=None) == -1 and rope(f=None) == -1
    assert rope(T=-1) == -1 and rope(H=0) == -1 and rope(H=65536) == -1
    assert rope(xs=neg) == -1 and rope(os=neg) == -1
    assert rope(x=17) == -1 and rope(dtype=2, x=18) == -1 and rope(pos=20, flags=4) == -1 and b"aligned" in err()
    assert rope(x=32, out=32, os=odd) == -1 and b"strides of x" in err()
    assert rope(T=0, x=None, out=None) == 0                        # nothing to do

    def slots(ptr=16, lens=16, b=2, table=16, bs=4, w=4, pages=8, T=4, s=16, p=16):
        return lib.mla_cache_slots(ptr, lens, b, table, bs, w, pages, T, s, p, None)
    assert slots(b=0) == -1 and slots(T=-1) == -1 and slots(w=0) == -1 and slots(bs=-1) == -1 and slots(pages=0) == -1
    assert slots(ptr=None) == -1 and slots(s=None) == -1 and slots(s=20) == -1
    assert slots(T=0, s=None) == 0

    def write(lat=16, ls=s2, rp=16, rs=s2, dtype=0, T=4, h=1, w=None, eps=1e-6, pos=None, f=None, m=1.0, flags=0, at=16,
              pool=16, pages=8, page=64):
        return lib.mla_cache_write(lat, ls, rp, rs, dtype, T, h, w, eps, pos, f, m, flags, at, pool, pages, page, None)
    assert write(page=32) == -2 and b"page_size" in err()
    assert write(dtype=-1) == -1 and write(flags=2) == -1 and write(h=0) == -1 and write(pages=0) == -1
    assert write(w=16, eps=-1.0) == -1 and b"eps" in err()
    assert write(f=16) == -1 and b"null" in err()                  # frequencies without positions
    assert write(ls=odd) == -1 and write(rs=neg) == -1 and b"multiples of 8" in err()
    assert write(lat=24) == -1 and write(w=24) == -1 and write(at=20) == -1 and b"aligned" in err()
    assert write(T=1 << 32) == -1 and b"2^31" in err()
    assert write(T=0, lat=None) == 0
    assert lib.mla_cache_write_fp8(16, s2, 16, s2, 0, 4, 1, None, 1e-6, None, None, 1.0, 0, 16, 16, None, 8, 64, None) == -1

    def read(pool=16, pages=8, page=64, h=1, at=16, T=4, out=16, os=s2):
        return lib.mla_cache_read(pool, pages, page, h, at, T, out, os, None)
    assert read(page=128) == -2 and read(pages=0) == -1 and read(pool=None) == -1 and read(out=24) == -1 and read(os=odd) == -1
    assert read(T=0, out=None) == 0
    assert lib.mla_cache_read_fp8(16, None, 8, 64, 1, 16, 4, 16, s2, None) == -1

    def verify(t=16, ts=s2, d=16, ds=s2, dtype=0, tok=16, u=16, un=16, n=None, b=2, s=3, V=9, acc=16, out=16):
        return lib.mla_verify_draft(t, ts, d, ds, dtype, tok, u, un, n, b, s, V, acc, out, None)
    assert verify(t=None) == -1 and verify(d=16, ds=None) == -1 and verify(un=None) == -1
    assert verify(b=0) == -1 and verify(s=0) == -1 and verify(V=0) == -1 and verify(dtype=7) == -1
    assert verify(ts=neg) == -1 and verify(ds=neg) == -1 and verify(tok=18) == -1 and b"aligned" in err()

    # the FP8 decode of any number of rows checks what the 16-row one checks, but for the rows
    s3 = (ctypes.c_int64 * 3)(576, 576, 576)

    def rows(h_q=128, d=576, dv=512, page=64, flags=0, k8=16, scale=0.04):
        return lib.mla_decode_paged_fp8_rows(16, s3, 1, 1, h_q, d, k8, 16, 1, page, 1, 16, 1, 16, dv, 16, 1, 16,
                                             ctypes.c_float(scale), 1, 16, 16, 256, 1 << 20, flags, None)
    assert rows(d=512) == -2 and rows(dv=256) == -2 and rows(page=32) == -2
    assert rows(flags=2) == -1 and rows(k8=None) == -1 and rows(scale=-1.0) == -1 and rows(k8=24) == -1


def test_frequency_refusals():
    for bad in (dict(dim=63), dict(dim=0), dict(base=1.0), dict(factor=0.5), dict(scaling="cubic"),
                dict(scaling="yarn", factor=4.0, beta_fast=1.0, beta_slow=2.0), dict(dim=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            ops.rope_frequencies(**bad)
    assert ops.rope_magnitude(1.0) == 1.0 and math.isclose(ops.rope_magnitude(40.0), 0.1 * math.log(40.0) + 1)


def test_written_tensors_that_need_a_gradient_are_refused():
    grad = lambda t: t.requires_grad_()
    calls = [
        (ops.mla_rope, rope_args(out=grad(z(5, 4, 64))), "out must not require"),
        (ops.mla_cache_write, write_args(k_cache=grad(z(3, 64, 1, 576))), "the cache must not require"),
        (ops.mla_cache_write_fp8, write_args(True, k_scale=grad(z(1, 3, 64, dtype=f32))), "k_scale must not require"),
        (ops.mla_cache_read, dict(k_cache=z(3, 64, 1, 576), slots=z(6, dtype=i64), out=grad(z(6, 1, 576))), "out must not require"),
    ]
    rows = dict(q=z(3, 1, 128, 576), k8=z(10, 64, 1, 576, dtype=torch.uint8), k_scale=z(1, 10, 64, dtype=f32),
                block_table=z(3, 6, dtype=i32), cache_seqlens=z(3, dtype=i32), dv=512, tile_metadata=z(5, 8, dtype=i32),
                num_splits=z(4, dtype=i32))
    calls += [(ops.mla_decode_paged_fp8_rows, dict(rows, out=grad(z(3, 1, 128, 512))), "out must not require"),
              (ops.mla_decode_paged_fp8_rows, dict(rows, lse=grad(z(3, 128, 1, dtype=f32))), "lse must not require")]
    for fn, kw, msg in calls:
        with pytest.raises(ValueError, match=msg):
            fn(**kw)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensor"):      # passes the checks
            fn(**kw)


def test_rope_refuses_what_it_cannot_differentiate():
    import torch.autograd.forward_ad as fwd
    freq = ops.rope_frequencies(64)
    with pytest.raises(ValueError, match="derivative by inv_freq"):
        ops.mla_rope(**rope_args(inv_freq=freq.clone().requires_grad_()))
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensor"):
        ops.mla_rope(**rope_args(inv_freq=freq.clone().requires_grad_()))
    with fwd.dual_level():
        with pytest.raises(ValueError, match="derivative by inv_freq"):
            ops.mla_rope(**rope_args(inv_freq=fwd.make_dual(freq, torch.ones_like(freq))))
        dual = fwd.make_dual(z(5, 4, 64), z(5, 4, 64))
        with pytest.raises(ValueError, match="needs a gradient"):
            ops.mla_rope(**rope_args(x=dual, out=z(5, 4, 64)))
        with pytest.raises(ValueError, match="CUDA tensor"):
            ops.mla_rope(**rope_args(x=dual))


def test_marshalling_module_is_rebuilt_for_another_torch(monkeypatch, tmp_path):
    made = []

    def compile_it(cmd, *a, **kw):
        made.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B.subprocess, "check_call", compile_it)
    B._build_binding(False)
    B._build_binding(False)
    assert len(made) == 1
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    B._build_binding(False)
    B._build_binding(False)
    assert len(made) == 2


def test_slots_refuses_outputs_among_its_arguments():
    words = z(64, dtype=i32)
    a = dict(block_table=words[:12].view(3, 4), cache_seqlens=words[12:15], row_ptr=words[15:19], num_pages=12, tokens=3)
    for name, at in (("positions", 14), ("positions", 9), ("positions", 17)):
        with pytest.raises(ValueError, match="positions must not overlap the arguments"):
            ops.mla_cache_slots(**a, **{name: words[at:at + 3]})
    with pytest.raises(ValueError, match="slots must not overlap the arguments"):
        ops.mla_cache_slots(**a, slots=words[18:24].view(i64))
    with pytest.raises(ValueError, match="slots and positions"):
        ops.mla_cache_slots(**a, slots=words[24:30].view(i64), positions=words[29:32])
    with pytest.raises(ValueError, match="CUDA tensor"):               # beside them is in order
        ops.mla_cache_slots(**a, slots=words[20:26].view(i64), positions=words[26:29])


def test_decode_rows_refuses_outputs_among_its_arguments():
    q = z(3, 1, 128, 576)
    a = dict(q=q, k8=z(10, 64, 1, 576, dtype=torch.uint8), k_scale=z(1, 10, 64, dtype=f32),
             block_table=z(3, 6, dtype=i32), cache_seqlens=z(3, dtype=i32), dv=512, tile_metadata=z(5, 8, dtype=i32),
             num_splits=z(4, dtype=i32))
    inside = q.view(-1)[:3 * 128 * 512].view(3, 1, 128, 512)
    with pytest.raises(ValueError, match="out must not overlap the arguments"):
        ops.mla_decode_paged_fp8_rows(**a, out=inside)
    with pytest.raises(ValueError, match="lse must not overlap the arguments"):
        ops.mla_decode_paged_fp8_rows(**a, lse=a["k_scale"].view(-1)[:384].view(3, 128, 1))
    both = z(3 * 128 * 512 + 2 * 384)
    out, lse = both[:3 * 128 * 512].view(3, 1, 128, 512), both[-768:].view(f32).view(3, 128, 1)
    with pytest.raises(ValueError, match="out and lse"):
        ops.mla_decode_paged_fp8_rows(**a, out=out, lse=both[:768].view(f32).view(3, 128, 1))
    with pytest.raises(ValueError, match="CUDA tensor"):               # beside each other is in order
        ops.mla_decode_paged_fp8_rows(**a, out=out, lse=lse)


def test_capture_is_looked_for_on_the_tensors_device(monkeypatch):
    current = [0]

    class on:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[0] == 1)
    assert ops._capturing(torch.device("cuda", 1)) and current == [0]
    assert not ops._capturing(torch.device("cuda", 0))


def test_captured_calls_have_scratch_of_their_own(monkeypatch):
    class Stream:
        cuda_stream = 7

    capturing = [False]
    monkeypatch.setattr(ops, "_ws_cache", {})
    monkeypatch.setattr(ops, "_capturing", lambda device: capturing[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    cpu = torch.device("cpu")
    shared = ops._default_workspace(1000, cpu)
    assert ops._default_workspace(900, cpu) is shared
    capturing[0] = True
    first, second = ops._default_workspace(900, cpu), ops._default_workspace(5000, cpu)
    assert first is not shared and second is not first and first.numel() >= 900 and second.numel() >= 5000
    assert not first[:256].any() and not second[:256].any()        # the status block
    capturing[0] = False
    assert ops._default_workspace(900, cpu) is shared              # neither replaced nor freed


def test_written_tensors_that_carry_a_tangent_are_refused():
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level():
        dual = lambda *shape: fwd.make_dual(z(*shape), z(*shape))
        for fn, kw in ((ops.mla_rope, rope_args(out=dual(5, 4, 64))),
                       (ops.mla_cache_write, write_args(k_cache=dual(3, 64, 1, 576))),
                       (ops.mla_cache_read, dict(k_cache=z(3, 64, 1, 576), slots=z(6, dtype=i64), out=dual(6, 1, 576)))):
            with pytest.raises(ValueError, match="carry a tangent"):
                fn(**kw)
