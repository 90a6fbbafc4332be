"""The operators together, as one training step of a small mixture-of-experts
model over simulated ranks uses them: gate -> split counts -> all-to-all ->
experts -> all-to-all back -> all-reduce with dropout and residual -> cross
entropy over the vocabulary pieces -> gradients -> ZeRO-1 step.  Everything is
compared with the same step in 64 bits; the step runs eagerly and, from the
all-reduce on, captured in a graph."""
import pytest
import torch

pytestmark = pytest.mark.gpu
HALF = torch.finfo(torch.bfloat16).eps / 2  # half a step of bf16


@pytest.fixture(scope="module")
def rc():
    import collective_rc_all_b200 as m
    assert torch.cuda.is_available()
    return m


P, T, D, E, K, V = 4, 96, 64, 8, 2, 1003   # ranks, tokens per rank, width, experts (two per rank), top k, vocabulary


def ranks(f):
    return [f(r) for r in range(P)]


def dispatch_order(ids):
    """Rows of a rank's (token, slot) pairs in expert order, and the counts per destination rank."""
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    order = order[flat[order] >= 0]
    dest = torch.div(flat[order], E // P, rounding_mode="floor")
    return order, torch.bincount(dest, minlength=P)


def test_moe_training_step(rc):
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = ranks(lambda r: rnd(T, D).bfloat16())
    mask = ranks(lambda r: (torch.rand(T, generator=g, device="cuda") > 0.1).to(torch.uint8))
    logits = ranks(lambda r: rnd(T, E))
    expert_scale = 0.5 + torch.rand(E, generator=g, device="cuda")          # expert e multiplies its tokens by this

    # gate
    ids = ranks(lambda r: torch.empty(T, K, dtype=torch.int32, device="cuda"))
    w = ranks(lambda r: torch.empty(T, K, device="cuda"))
    counts = ranks(lambda r: torch.empty(E, dtype=torch.int32, device="cuda"))
    stats, balance = torch.empty(2 * E + 1, device="cuda"), torch.empty(1, device="cuda")
    rc.rc_moe_gate(logits, ids, w, counts, stats, balance, token_mask=mask, coef=0.1)

    # dispatch by the counts, expert, combine
    per_dest = torch.stack(counts).view(P, P, E // P).sum(2)
    split = per_dest.cpu().numpy()
    orders = [dispatch_order(i) for i in ids]
    for r in range(P):
        assert torch.equal(orders[r][1], per_dest[r].long())                # the gate's counts are the split counts
    send = [x[r][torch.div(o, K, rounding_mode="floor")].contiguous() for r, (o, _) in enumerate(orders)]
    recv = [torch.empty(int(split[:, q].sum()), D, dtype=torch.bfloat16, device="cuda") for q in range(P)]
    rc.rc_all_to_all_v([s.view(-1) for s in send], [t.view(-1) for t in recv], split * D)
    tags = [ids[r].reshape(-1)[o].int() for r, (o, _) in enumerate(orders)]
    tag_recv = [torch.empty(int(split[:, q].sum()), dtype=torch.int32, device="cuda") for q in range(P)]
    rc.rc_all_to_all_v(tags, tag_recv, split)
    for q in range(P):
        assert bool((torch.div(tag_recv[q], E // P, rounding_mode="floor") == q).all())  # every token reached its expert's rank
        recv[q] = (recv[q].float() * expert_scale[tag_recv[q].long()][:, None]).bfloat16()
    back = [torch.empty_like(s) for s in send]
    rc.rc_all_to_all_v([t.view(-1) for t in recv], [b.view(-1) for b in back], (split * D).T)
    part = []
    for r in range(P):
        y = torch.zeros(T * K, D, device="cuda")
        y[orders[r][0]] = back[r].float()
        part.append((y.view(T, K, D) * w[r][..., None]).sum(1).bfloat16())

    # row-parallel end of a layer: the ranks' parts are summed, dropped, added to the residual
    base = rnd(T, D).bfloat16()
    res = ranks(lambda r: base.clone())
    h = ranks(lambda r: torch.empty_like(base))
    prob, seed, offset = 0.2, 1234567, 4096
    wv = [t.contiguous() for t in torch.split((rnd(V, D) / 8).bfloat16(), [min(V, (r + 1) * -(-V // P)) - r * -(-V // P) for r in range(P)])]
    y = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    y[::9] = -100
    live = y >= 0
    dloss = live.float() / live.sum()
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dh, dw = torch.empty_like(base), [torch.empty_like(t) for t in wv]
    dpart = ranks(lambda r: torch.empty_like(base))
    ws = torch.empty(rc.rc_vocab_ce_workspace(T, D, V, P, backward=True), dtype=torch.uint8, device="cuda")

    def tail():
        rc.rc_all_reduce_dropout(part, h, prob, seed, offset=offset, residual=res)
        rc.rc_vocab_ce_forward(h[0], wv, y, loss, lse, workspace=ws)
        rc.rc_vocab_ce_backward(h[0], wv, y, lse, dloss, dh, dw, workspace=ws)
        rc.rc_dropout([dh] * P, dpart, prob, seed, offset=offset)

    tail()
    rc.rc_stream_status()

    # the same in 64 bits, from the parts on
    ones = torch.ones(T * D, device="cuda")
    kept = torch.empty_like(ones)
    rc.rc_dropout([ones], [kept], prob, seed, offset=offset)
    factor = 65536 / (65536 - round(prob * 65536))
    assert bool(((kept == 0) | ((kept.double() - factor).abs() < 1e-6)).all())
    m = (kept != 0).double().view(T, D) * factor
    want = base.double() + m * torch.stack(part).double().sum(0)
    # the fold is in binary32 (p terms), the result rounded once
    room = P * 2.0 ** -23 * torch.stack(part).double().abs().sum(0) * factor
    for r in range(P):
        assert bool(((h[r].double() - want).abs() <= HALF * (want.abs() + room) + room).all())
        assert torch.equal(h[r], h[0])
    z = h[0].double() @ torch.cat(wv).double().T
    lse64 = torch.logsumexp(z, 1)
    loss64 = torch.where(live, lse64 - z.gather(1, torch.where(live, y, 0).long()[:, None])[:, 0], 0.0)
    # d = 64: a few sums of 16 products in binary32, an exponential and a logarithm
    assert float((loss.double() - loss64).abs().max()) <= 1e-5
    G = torch.softmax(z, 1)
    G[live, y[live].long()] -= 1
    G *= torch.where(live, dloss.double(), 0.0)[:, None]
    for got, ref in ((dh, G @ torch.cat(wv).double()), (torch.cat(dw), G.T @ h[0].double())):
        # G in two planes (2^-16), the result one rounding: together below half a step and a little
        assert float((got.double() - ref).norm()) <= 1.02 * HALF * float(ref.norm())
    for r in range(P):
        assert torch.equal(dpart[r], (dh.float() * kept.view(T, D)).bfloat16())

    # captured: the same bits, also after the inputs changed and changed back
    first = [t.clone() for t in (h[1], loss, lse, dh, *dw, *dpart)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tail()
    saved = [t.clone() for t in part]
    for t in part:
        t.mul_(2)
    graph.replay()
    for t, s in zip(part, saved):
        t.copy_(s)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (h[1], loss, lse, dh, *dw, *dpart)))

    # router gradient, and the optimizer on the head's gradient (one shard per rank, the gradients replicated here)
    dlogits = ranks(lambda r: torch.empty_like(logits[r]))
    dweights = ranks(lambda r: torch.ones(T, K, device="cuda"))
    rc.rc_moe_gate_backward(logits, ids, stats, dlogits, dweights=dweights, dloss=torch.ones(1, device="cuda"), token_mask=mask, coef=0.1)
    for r in range(P):
        # weights sum to one, so a constant upstream leaves the balance term alone
        pr = torch.softmax(logits[r].double(), 1)
        a = 0.1 * E * stats[:E].double() / float(stats[2 * E])
        ref = torch.where(mask[r][:, None] != 0, pr * (a - (pr * a).sum(1, keepdim=True)), 0.0)
        assert float((dlogits[r].double() - ref).abs().max()) <= 1e-6
    flat = torch.cat([t.reshape(-1) for t in dw])
    n = flat.numel() // P * P
    grads = ranks(lambda r: flat[:n].clone())
    master = ranks(lambda r: torch.cat([t.reshape(-1) for t in wv])[:n].float().view(P, -1)[r].clone())
    before = [t.clone() for t in master]
    m1, m2 = ranks(lambda r: torch.zeros(n // P, device="cuda")), ranks(lambda r: torch.zeros(n // P, device="cuda"))
    params = ranks(lambda r: torch.empty(n, dtype=torch.bfloat16, device="cuda"))
    rc.rc_zero1_step(grads, params, master, m1, m2, lr=1e-3)
    rc.rc_stream_status()
    for r in range(P):
        assert torch.equal(params[r], torch.cat(master).bfloat16())
        moved = grads[0].view(P, -1)[r] != 0
        assert bool((master[r] != before[r])[moved].float().mean() > 0.9)
