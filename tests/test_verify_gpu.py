"""Verification of drafted tokens (mla_verify_draft) against the rule written out in fp64, one
sequence after another.  Results are whole numbers and must be equal."""

import ctypes

import numpy as np
import pytest
import torch

from paged_mla_decode_11_b200 import ops

pytestmark = pytest.mark.gpu


def weights(w):
    return np.where(np.isfinite(w) & (w > 0), w, 0.0)


def expected(target, tokens, u, u_new, draft=None, num=None):
    target = target.double().cpu().numpy()
    draft = None if draft is None else draft.double().cpu().numpy()
    tokens, u, u_new = tokens.cpu().numpy(), u.double().cpu().numpy(), u_new.double().cpu().numpy()
    b, s1, V = target.shape
    counts, made = [], np.full((b, s1), -1)
    for i in range(b):
        n = s1 - 1 if num is None else min(max(int(num[i]), 0), s1 - 1)
        r = 0
        while r < n:
            t = tokens[i, r]
            if not (0 <= t < V):
                break
            if not u[i, r] * (1.0 if draft is None else draft[i, r, t]) < target[i, r, t]:
                break
            made[i, r] = t
            r += 1
        counts.append(r)
        p = target[i, r]
        w = weights(p)
        if r < n:
            q = np.zeros(V)
            if draft is not None:
                q = draft[i, r]
            elif 0 <= tokens[i, r] < V:
                q[tokens[i, r]] = 1.0
            with np.errstate(invalid="ignore"):
                rest = weights(p - q)
            if rest.sum() > 0:
                w = rest
        if w.sum() > 0:
            c = np.cumsum(w)
            over = np.nonzero((c > max(u_new[i], 0.0) * c[-1]) & (w > 0))[0]
            made[i, r] = over[0] if len(over) else np.nonzero(w)[0][-1]
    return np.array(counts), made


def check(target, tokens, u, u_new, draft=None, num=None):
    got = ops.mla_verify_draft(target, tokens, u, u_new, draft_probs=draft, num_drafts=num)
    counts, made = expected(target, tokens, u, u_new, draft, None if num is None else num.cpu())
    np.testing.assert_array_equal(got[0].cpu().numpy(), counts)
    np.testing.assert_array_equal(got[1].cpu().numpy(), made)
    return counts, made


def draw(b, s, V, dtype, seed=0, noise=0.6):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = 3 * torch.randn(b, s + 1, V, generator=g, device="cuda")
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits[:, :s] + noise * torch.randn(b, s, V, generator=g, device="cuda"), -1)
    tokens = torch.multinomial(draft.reshape(b * s, V), 1, generator=g).view(b, s).to(torch.int32)
    return (target.to(dtype), tokens, torch.rand(b, s, generator=g, device="cuda"),
            torch.rand(b, generator=g, device="cuda"), draft.to(dtype))


@pytest.mark.parametrize("b,s,V", [(1, 1, 1), (1, 1, 2), (3, 2, 7), (1, 3, 32003), (5, 1, 511), (64, 3, 1000),
                                   (37, 8, 4097), (160, 2, 333), (300, 1, 129), (2, 40, 515), (1, 33, 8191)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_verify(b, s, V, dtype):
    target, tokens, u, u_new, draft = draw(b, s, V, dtype, seed=b + s + V)
    check(target, tokens, u, u_new, draft)
    check(target, tokens, u, u_new)
    num = torch.randint(-1, s + 2, (b,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.int32)
    check(target, tokens, u, u_new, draft, num)


def test_large_vocabulary_and_strided_rows():
    target, tokens, u, u_new, draft = draw(6, 3, 131072, torch.float32, seed=3)
    counts, _ = check(target, tokens, u, u_new, draft)
    assert 0 < counts.sum() < 18                             # both outcomes occur
    wide = torch.full((6, 5, 131073 + 40), float("nan"), device="cuda")
    wide[:, :4, 3:131072 + 3] = target
    check(wide[:, :4, 3:131072 + 3], tokens, u, u_new, draft)


def test_the_ends_of_the_uniform_range():
    target, tokens, u, u_new, draft = draw(8, 2, 999, torch.float32, seed=4)
    for v in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0):
        check(target, tokens, u, torch.full_like(u_new, v), draft)
    check(target, tokens, torch.zeros_like(u), u_new, draft)          # all accepted
    counts, _ = check(target, tokens, torch.full_like(u, 1e30), u_new, draft)
    assert (counts == 0).all()                                        # all rejected


def test_one_certain_token_and_zeros_around_it():
    V = 2000
    target = torch.zeros(4, 2, V, device="cuda")
    target[:, :, 1234] = 1.0
    draft = torch.zeros(4, 1, V, device="cuda")
    draft[:, 0, 77] = 1.0
    tokens = torch.tensor([[77], [1234], [77], [1234]], dtype=torch.int32, device="cuda")
    u = torch.tensor([[0.0], [0.0], [0.5], [0.9]], device="cuda")
    for v in (0.0, 0.3, 0.999999):
        counts, made = check(target, tokens, u, torch.full((4,), v, device="cuda"), draft)
        # draft probability 0 at 1234: accepted; 77 has target probability 0: rejected even with u = 0
        assert counts.tolist() == [0, 1, 0, 1] and (made[:, 0] == 1234).all()


def test_rows_that_leave_nothing():
    V = 1500
    target, tokens, u, u_new, draft = draw(5, 2, V, torch.float32, seed=7)
    target[0, 0] = draft[0, 0] * 0.5                 # p <= q everywhere: drawn from p when rejected
    u[0, 0] = 0.9
    target[1, 0] = 0                                 # nothing at all: -1
    target[2] = float("nan")
    target[3, 0, 5], target[3, 0, 6] = float("inf"), float("nan")
    draft[3, 0, 9] = float("nan")
    tokens[3, 0] = 9
    tokens[4, 0] = V                                 # outside the vocabulary
    counts, made = check(target, tokens, u, u_new, draft)
    assert counts[0] == 0 and made[0, 0] >= 0 and made[1, 0] == -1 and made[2, 0] == -1 and counts[4] == 0
    tokens[4, 0] = -5
    check(target, tokens, u, u_new)


def test_tokens_follow_the_targets_distribution():
    """Many uniform numbers on one small distribution: frequencies of the first token approach the
    target's probabilities whatever the draft's (here far from them)."""
    b, V = 20000, 6
    p = torch.tensor([0.30, 0.05, 0.25, 0.0, 0.15, 0.25], device="cuda")
    q = torch.tensor([0.05, 0.55, 0.10, 0.2, 0.05, 0.05], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(11)
    tokens = torch.multinomial(q.expand(b, V), 1, generator=g).to(torch.int32)
    _, made = ops.mla_verify_draft(p.expand(b, 2, V), tokens, torch.rand(b, 1, generator=g, device="cuda"),
                                   torch.rand(b, generator=g, device="cuda"), draft_probs=q.expand(b, 1, V))
    seen = torch.bincount(made[:, 0].long(), minlength=V).double() / b
    # five standard deviations of a frequency over b draws
    assert ((seen.cpu() - p.double().cpu()).abs() <= 5 * (p.double().cpu() * (1 - p.double().cpu()) / b).sqrt()).all()


def test_streams_graphs_and_repeats():
    target, tokens, u, u_new, draft = draw(16, 3, 5000, torch.bfloat16, seed=12)
    want = ops.mla_verify_draft(target, tokens, u, u_new, draft_probs=draft)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ops.mla_verify_draft(target, tokens, u, u_new, draft_probs=draft)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = ops.mla_verify_draft(target, tokens, u, u_new, draft_probs=draft)
    for seed in (13, 14):
        new = draw(16, 3, 5000, torch.bfloat16, seed=seed)
        for dst, src in zip((target, tokens, u, u_new, draft), new):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        counts, made = expected(*new)
        np.testing.assert_array_equal(held[0].cpu().numpy(), counts)
        np.testing.assert_array_equal(held[1].cpu().numpy(), made)


def limited(args, timeout_ns, missing):
    """mla_verify_draft_selftest on the arguments of mla_verify_draft (with draft rows)."""
    target, tokens, u, u_new, draft = args
    b, s1, V = target.shape
    accepted = torch.full((b,), 7, dtype=torch.int32, device="cuda")
    made = torch.full((b, s1), 7, dtype=torch.int32, device="cuda")
    strides = [(ctypes.c_int64 * 2)(t.stride(0), t.stride(1)) for t in (target, draft)]
    kind = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}[target.dtype]
    rc = ops.load_library().mla_verify_draft_selftest(
        target.data_ptr(), strides[0], draft.data_ptr(), strides[1], kind, tokens.data_ptr(), u.data_ptr(),
        u_new.data_ptr(), None, b, s1 - 1, V, accepted.data_ptr(), made.data_ptr(), timeout_ns, missing,
        torch.cuda.current_stream().cuda_stream)
    assert rc == ops.MLA_OK
    torch.cuda.synchronize()
    return accepted, made


@pytest.mark.parametrize("b,s,V", [(1, 1, 32003), (5, 3, 131072), (64, 3, 4096), (300, 1, 129)])
def test_sums_that_do_not_arrive_leave_no_result(b, s, V):
    # 2 ms of waiting for one sum that nobody sends: no token is made up, and the next call is as ever
    args = draw(b, s, V, torch.float32, seed=b)
    accepted, made = limited(args, 2_000_000, 1)
    assert (accepted == -1).all() and (made == -1).all()
    target, tokens, u, u_new, draft = args
    check(target, tokens, u, u_new, draft)


@pytest.mark.parametrize("b,s,V", [(1, 1, 32003), (5, 3, 131072), (64, 3, 4096), (300, 1, 129), (100, 2, 50000)])
def test_waits_that_give_up_early_change_nothing(b, s, V):
    # a limit of zero: waits give up while other CTAs still sum, meet them, and find the sums
    args = draw(b, s, V, torch.float32, seed=b + 1)
    target, tokens, u, u_new, draft = args
    target[0, 0] = draft[0, 0] * 0.5                 # nothing left after a rejection: a second exchange
    u[0, 0] = 0.9
    counts, made = expected(*args)
    for _ in range(20):
        got = limited(args, 0, 0)
        np.testing.assert_array_equal(got[0].cpu().numpy(), counts)
        np.testing.assert_array_equal(got[1].cpu().numpy(), made)
