"""What autograd knows of the tensors that the operators of a serving step write: their versions
advance, so a backward pass that saved one of them raises instead of using the new values."""

import pytest
import torch

from paged_mla_decode_11_b200 import ops

pytestmark = pytest.mark.gpu

CHANGED = "modified by an inplace operation"


def plan(b=3, width=4):
    table = torch.arange(b * width, dtype=torch.int32, device="cuda").view(b, width)
    lens = torch.tensor([5, 70, 130], dtype=torch.int32, device="cuda")
    ptr = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device="cuda")
    return table, lens, ptr


def test_positions_reused_before_the_backward_pass():
    table, lens, ptr = plan()
    slots, pos = ops.mla_cache_slots(table, lens, ptr, 12, 6)
    freq = ops.rope_frequencies(64, device="cuda")
    x = torch.randn(6, 4, 64, device="cuda", requires_grad=True)
    y = ops.mla_rope(x, pos, freq)
    ops.mla_cache_slots(table, lens + 1, ptr, 12, 6, slots=slots, positions=pos)     # the next step's
    with pytest.raises(RuntimeError, match=CHANGED):
        y.sum().backward()


def test_input_of_a_product_rotated_in_place():
    freq, pos = ops.rope_frequencies(64, device="cuda"), torch.arange(6, device="cuda")
    x, w = torch.randn(6, 4, 64, device="cuda"), torch.randn(64, 8, device="cuda", requires_grad=True)
    y = x @ w
    ops.mla_rope(x, pos, freq, out=x)
    with pytest.raises(RuntimeError, match=CHANGED):
        y.sum().backward()
    # a fresh output leaves what was saved
    y = x @ w
    ops.mla_rope(x, pos, freq)
    y.sum().backward()


def test_versions_of_all_written_tensors():
    table, lens, ptr = plan()
    freq = ops.rope_frequencies(64, device="cuda")
    both = torch.randn(6, 1, 576, device="cuda").to(torch.bfloat16)
    slots, pos = torch.zeros(6, dtype=torch.int64, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")
    pool = torch.zeros(12, 64, 1, 576, dtype=torch.bfloat16, device="cuda")
    k8, ks = torch.zeros(12, 64, 1, 576, dtype=torch.uint8, device="cuda"), torch.ones(1, 12, 64, device="cuda")
    rows, q = torch.empty_like(both), torch.randn(3, 2, 64, 576, device="cuda").to(torch.bfloat16)
    out, lse = torch.empty(3, 2, 64, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 64, 2, device="cuda")
    tile, splits = ops.get_mla_metadata(lens, 128, 1)
    turned = torch.empty_like(both)
    steps = [
        (lambda: ops.mla_cache_slots(table, lens, ptr, 12, 6, slots=slots, positions=pos), (slots, pos), (table, lens, ptr)),
        (lambda: ops.mla_rope(both, pos, freq, out=turned), (turned,), (both, pos, freq)),
        (lambda: ops.mla_cache_write(both[..., :512], both[..., 512:], slots, pool), (pool,), (both, slots)),
        (lambda: ops.mla_cache_write_fp8(both[..., :512], both[..., 512:], slots, k8, ks), (k8, ks), (both, slots)),
        (lambda: ops.mla_cache_read(pool, slots, out=rows), (rows,), (pool, slots)),
        (lambda: ops.mla_cache_read_fp8(k8, ks, slots, out=rows), (rows,), (k8, ks, slots)),
        (lambda: ops.mla_decode_paged_fp8_rows(q, k8, ks, table, lens, 512, tile, splits, out=out, lse=lse), (out, lse),
         (q, k8, ks, table, lens, tile, splits)),
    ]
    for call, changed, kept in steps:
        before = [t._version for t in changed], [t._version for t in kept]
        call()
        assert all(t._version > v for t, v in zip(changed, before[0]))
        assert [t._version for t in kept] == before[1]
    with torch.inference_mode():                     # tensors without a version
        pool = torch.zeros(12, 64, 1, 576, dtype=torch.bfloat16, device="cuda")
        ops.mla_cache_write(both[..., :512], both[..., 512:], slots, pool)
    ops.mla_cache_write(both[..., :512], both[..., 512:], slots, pool)
    assert torch.equal(ops.mla_cache_read(pool, slots), both)
