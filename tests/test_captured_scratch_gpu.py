"""Decodes captured without a workspace: their scratch belongs to the graph.  A larger call on the
same stream replaces the stream's shared buffer; replays must neither use the freed memory nor
disturb what lies there now."""

import pytest
import torch

from paged_mla_decode_11_b200 import ops
from paged_mla_decode_11_b200 import workloads as W

pytestmark = pytest.mark.gpu


def decode(kind, h_q, lens, seed):
    """A call without workspace, and its result from a call with one."""
    if kind == "sparse":
        x = W.make_inputs_sparse(W.custom(len(lens), 1, h_q, 1, lens, causal=True), topk=600, seed=seed)
    elif kind == "bf16":
        x = W.make_inputs(W.custom(len(lens), 1, h_q, 1, lens, causal=True), seed=seed)
    else:
        x = W.make_inputs_fp8(W.custom(len(lens), 1, h_q, 1, lens, causal=True), seed=seed)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    if kind == "sparse":
        tile, splits = ops.get_mla_metadata_csr(d["row_ptr"], h_q, 1)
        call = lambda **kw: ops.mla_decode_sparse(d["q"], d["k_cache"], d["block_table"], d["cache_seqlens"], d["row_ptr"],
                                                  d["col_idx"], 512, tile, splits, causal=True, **kw)
    else:
        tile, splits = ops.get_mla_metadata(d["cache_seqlens"], h_q, 1)
        if kind == "bf16":
            call = lambda **kw: ops.mla_decode_paged(d["q"], d["k_cache"], d["block_table"], d["cache_seqlens"], 512, tile,
                                                     splits, causal=True, **kw)
        else:
            fn = ops.mla_decode_paged_fp8 if h_q <= 16 else ops.mla_decode_paged_fp8_rows
            call = lambda **kw: fn(d["q"], d["k8"], d["k_scale"], d["block_table"], d["cache_seqlens"], 512, tile, splits,
                                   causal=True, **kw)
    ws = ops.new_workspace(ops.workspace_size(len(lens), 1, h_q, 1, tile.shape[0]), "cuda")
    want = call(workspace=ws)
    return call, want


@pytest.mark.parametrize("kind,h_q", [("bf16", 16), ("bf16", 128), ("fp8", 16), ("fp8", 128), ("sparse", 16)])
def test_larger_call_after_a_capture(kind, h_q):
    small, want = decode(kind, h_q, [3000, 1, 500], seed=1)
    large, want_large = decode(kind, h_q, [700] * 40, seed=2)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        small()                                              # the stream's buffer, of this size
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = small()
    with torch.cuda.stream(stream):
        got_large = large()                                  # a larger one takes its place
        junk = [torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda") for n in (1 << 20, 1 << 22, 1 << 24, 1 << 25)]
        graph.replay()
    torch.cuda.synchronize()
    for a, b in ((got, want), (got_large, want_large)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert all((j == 0x5a).all() for j in junk)
