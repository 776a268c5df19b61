"""One speculative serving step through the operators together, as a latent-attention model calls
them for a layer: prompt into the FP8 cache, then three tokens per sequence (one known, two
drafted) -- slots, cache write with norm and rotation, rotary queries, absorption, decode,
absorption, and the verification of the drafts against the step's probabilities.  Eager and as a
captured graph replayed on other inputs; compared with the layer written out in fp64 over the
per-head keys and values of the stored cache."""

import pytest
import torch

from paged_mla_decode_11_b200 import ops
from test_verify_gpu import expected

pytestmark = pytest.mark.gpu

B, NEW, H, V = 5, 3, 24, 2000
PREFIX = [0, 61, 64, 130, 700]
FREQ = dict(scaling="yarn", factor=40.0)


def draw(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)
    T = B * NEW
    d = dict(prompt=r(sum(PREFIX), 1, 576), kv=r(T, 1, 576), q=r(T, H, 192), head=r(H * 128, V, std=0.15))
    d["drafts"] = torch.randint(0, V, (B, NEW - 1), generator=g, device="cuda").to(torch.int32)
    d["draft_probs"] = torch.softmax(torch.randn(B, NEW - 1, V, generator=g, device="cuda"), -1)
    d["u"], d["u_new"] = torch.rand(B, NEW - 1, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    return d


def weights():
    g = torch.Generator(device="cuda").manual_seed(99)
    r = lambda *s, std: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)
    return dict(uk=r(H, 128, 512, std=128 ** -0.5), uv=r(H, 128, 512, std=512 ** -0.5),
                norm=(1 + 0.1 * torch.randn(512, generator=g, device="cuda")).to(torch.bfloat16))


class Layer:
    def __init__(self):
        self.w = weights()
        self.lens0 = torch.tensor(PREFIX, dtype=torch.int32, device="cuda")
        self.lens = self.lens0 + NEW
        width = -(-(max(PREFIX) + NEW) // 64)
        pages = B * width
        self.table = torch.randperm(pages, generator=torch.Generator().manual_seed(5)).to(torch.int32).view(B, width).cuda()
        self.k8 = torch.zeros(pages, 64, 1, 576, dtype=torch.float8_e4m3fn, device="cuda")
        self.scale = torch.ones(1, pages, 64, device="cuda")
        self.freq = ops.rope_frequencies(64, device="cuda", **FREQ)
        self.mag = ops.rope_magnitude(40.0)
        ptr = torch.zeros(B + 1, dtype=torch.int32)
        ptr[1:] = torch.tensor(PREFIX).cumsum(0)
        self.ptr0 = ptr.cuda()
        self.ptr = torch.arange(0, B * NEW + 1, NEW, dtype=torch.int32, device="cuda")
        self.softmax_scale = 192 ** -0.5

    def write(self, rows, lens, ptr):
        slots, pos = ops.mla_cache_slots(self.table, lens, ptr, self.k8.shape[0], rows.shape[0])
        ops.mla_cache_write_fp8(rows[..., :512], rows[..., 512:], slots, self.k8, self.scale, norm_weight=self.w["norm"],
                                positions=pos, inv_freq=self.freq, magnitude=self.mag)
        return pos

    def step(self, d):
        self.write(d["prompt"], self.lens0, self.ptr0)
        pos = self.write(d["kv"], self.lens, self.ptr)
        q_rope = ops.mla_rope(d["q"][..., 128:], pos, self.freq, magnitude=self.mag)
        q = ops.absorb_query(d["q"][..., :128], q_rope, self.w["uk"]).view(B, NEW, H, 576)
        plan, splits = ops.get_mla_metadata(self.lens, NEW * H, 1)
        lat, _ = ops.mla_decode_paged_fp8_rows(q, self.k8, self.scale, self.table, self.lens, 512, plan, splits,
                                               softmax_scale=self.softmax_scale, causal=True)
        o = ops.absorb_output(lat.view(B * NEW, H, 512), self.w["uv"])
        probs = torch.softmax((o.reshape(B, NEW, H * 128) @ d["head"]).float(), -1)
        accepted, tokens = ops.mla_verify_draft(probs, d["drafts"], d["u"], d["u_new"], draft_probs=d["draft_probs"])
        return o, probs, accepted, tokens

    def reference(self, d):
        """o in fp64, and the relative error its bf16 stages may add (2-norm)."""
        out, worst = torch.zeros(B * NEW, H, 128, dtype=torch.float64, device="cuda"), 0.0
        uk, uv = self.w["uk"].double(), self.w["uv"].double()
        turn = self.freq.double()
        for b in range(B):
            L = PREFIX[b] + NEW
            used = self.table[b, :-(-L // 64)].long()
            rows = (self.k8[used].float().double() * self.scale[0, used].double()[..., None, None]).flatten(0, 1)[:L, 0]
            # what was stored is the layer's row: normalised latent and rotated rope columns, to E4M3's half step
            raw = torch.cat([d["prompt"][int(self.ptr0[b]):int(self.ptr0[b + 1]), 0], d["kv"][b * NEW:(b + 1) * NEW, 0]]).double()
            a = torch.arange(L, device="cuda", dtype=torch.float64)[:, None] * turn
            rot = torch.stack([raw[:, 512::2] * a.cos() - raw[:, 513::2] * a.sin(),
                               raw[:, 512::2] * a.sin() + raw[:, 513::2] * a.cos()], -1).flatten(1) * self.mag
            lat = raw[:, :512] * torch.rsqrt(raw[:, :512].square().mean(-1, keepdim=True) + 1e-6) * self.w["norm"].double()
            want = torch.cat([lat, rot], -1)
            amax = want.abs().amax(-1, keepdim=True)
            assert ((rows - want).abs() <= 1.001 * torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * amax / 448) + 1e-5 * amax).all()
            for s in range(NEW):
                n = L - (NEW - 1 - s)
                q = d["q"][b * NEW + s].double()
                x0, x1 = q[:, 128::2], q[:, 129::2]
                a1 = (L - NEW + s) * turn
                qr = torch.stack([x0 * a1.cos() - x1 * a1.sin(), x0 * a1.sin() + x1 * a1.cos()], -1).flatten(1) * self.mag
                full = torch.cat([torch.einsum("hd,hdc->hc", q[:, :128], uk), qr], -1)
                x = full @ rows[:n].t() * self.softmax_scale
                p = torch.softmax(x, -1)
                out[b * NEW + s] = torch.einsum("hn,nc,hdc->hd", p, rows[:n, :512], uv)
                # rounding the absorbed query to bf16 moves a score by at most 2^-8 of its terms' sizes;
                # random signs leave their root sum of squares
                worst = max(worst, float((2.0 ** -8 * self.softmax_scale * (full.square() @ rows[:n].square().t()).sqrt()).max()))
        return out, 2 * worst + 4 * 2.0 ** -8


def check(layer, d, o, probs, accepted, tokens):
    ref, bound = layer.reference(d)
    assert (o.double() - ref).norm() <= bound * ref.norm()
    counts, made = expected(probs, d["drafts"], d["u"], d["u_new"], d["draft_probs"])
    assert accepted.tolist() == counts.tolist() and tokens.tolist() == made.tolist()


def test_step():
    layer, d = Layer(), draw(1)
    check(layer, d, *layer.step(d))


def test_captured_step():
    layer, d = Layer(), draw(2)
    layer.step(d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.step(d)
    for seed in (3, 4):
        for k, v in draw(seed).items():
            d[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        check(layer, d, *got)


def test_a_prefix_read_back_is_what_was_written():
    layer, d = Layer(), draw(5)
    layer.write(d["prompt"], layer.lens0, layer.ptr0)
    slots, _ = ops.mla_cache_slots(layer.table, layer.lens0, layer.ptr0, layer.k8.shape[0], sum(PREFIX) + 7)
    back = ops.mla_cache_read_fp8(layer.k8, layer.scale, slots)
    assert (back[sum(PREFIX):] == 0).all()                        # padding tokens
    bf16 = torch.zeros(layer.k8.shape, dtype=torch.bfloat16, device="cuda")
    rows = d["prompt"]
    ops.mla_cache_write(rows[..., :512], rows[..., 512:], slots[:sum(PREFIX)], bf16, norm_weight=layer.w["norm"],
                        positions=ops.mla_cache_slots(layer.table, layer.lens0, layer.ptr0, 10 ** 4, sum(PREFIX))[1],
                        inv_freq=layer.freq, magnitude=layer.mag)
    exact = ops.mla_cache_read(bf16, slots[:sum(PREFIX)])
    a, b = back[:sum(PREFIX)].double(), exact.double()
    amax = b.abs().amax(-1, keepdim=True)
    # E4M3's half step, and both sides' bf16 roundings
    assert ((a - b).abs() <= 1.001 * torch.maximum(2.0 ** -4 * b.abs(), 2.0 ** -10 * amax / 448) + 2.0 ** -7 * b.abs() + 1e-5 * amax).all()
